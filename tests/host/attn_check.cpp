// Host test of the attention operators' launch layer, built like api_check.cpp
// (tests/test_host_attention.py): kernel launches are recorded, not run.
// Checks, over small, odd, empty and largest sizes:
//   * the workspace query agrees with what the call accepts;
//   * the workgroups launched are those of the kernel's grid, each dispatch
//     within the cap on work-items, with and without a lowered cap;
//   * an axis without entries launches what its outputs need and no more;
//   * a failed launch ends the call with PC_ERR_HIP.
// Prints one line per failed check; exit status 0 when all pass.
#include <stdio.h>
#include <string.h>

#include <string>

#include "hip_stub.hpp"
#include "pc.h"

namespace {

int g_fails = 0;
#define CHECK(cond)                                                           \
    do {                                                                      \
        if (!(cond)) {                                                        \
            fprintf(stderr, "%s:%d: CHECK failed: %s\n", __FILE__, __LINE__, #cond); \
            ++g_fails;                                                        \
        }                                                                     \
    } while (0)

char *const F = reinterpret_cast<char *>(uintptr_t(1) << 20);
float *const FF = reinterpret_cast<float *>(F);

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

pc_attention sizes(int dtype, int n_kv, int group, int lq, int lk, int h, int hk, int d) {
    const pc_strides q = {int64_t(lq) * h * d, int64_t(h) * d, d}, k = {int64_t(lk) * hk * d, int64_t(hk) * d, d};
    return pc_attention{dtype, n_kv, group, lq, lk, h, hk, d, 0.1f, q, k, k, q, q, q, k, k};
}

// Workgroups of all launches whose kernel's name holds `name`; every dispatch within `cap` work-items.
int64_t groups(const char *name, uint64_t cap) {
    int64_t n = 0;
    for (const auto &l : stub::launches) {
        if (l.kernel.find(name) == std::string::npos) continue;
        CHECK(l.grid > 0 && l.grid_yz == 1);
        CHECK(uint64_t(l.grid) * l.block <= cap || l.grid == 1);
        n += l.grid;
    }
    return n;
}

void attention(int dtype, int n_kv, int group, int lq, int lk, int h, int hk, int d, uint64_t cap) {
    const pc_attention a = sizes(dtype, n_kv, group, lq, lk, h, hk, d);
    const int64_t pairs = int64_t(n_kv) * hk, rows = int64_t(group) * lq * (h / hk);
    int64_t need[2] = {-1, -1};
    for (int b = 0; b < 2; ++b) {
        CHECK(pc_cross_attention_workspace(&a, b, &need[b]) == PC_OK);
        CHECK(need[b] >= 0 && need[b] % 16 == 0);
    }
    stub::reset();
    CHECK(pc_cross_attention(&a, F, F, F, nullptr, nullptr, F, FF, need[0] ? F : nullptr, need[0], nullptr) == PC_OK);
    const int64_t fwd = groups("k_attn_fwd", cap), join = groups("k_attn_join", cap);
    if (pairs == 0 || rows == 0) {
        CHECK(stub::launches.empty());
    } else {
        const int64_t t128 = pairs * up(rows, 128), t256 = pairs * up(rows, 256);
        CHECK(fwd > 0 && (fwd % t128 == 0 || fwd == t256));
        CHECK((join > 0) == (need[0] > 0));
        if (join) CHECK(join == up(pairs * rows * (d / 4), 256) && fwd >= 2 * t128);
        if (join) {  // one byte less is refused, with nothing launched
            stub::reset();
            CHECK(pc_cross_attention(&a, F, F, F, nullptr, nullptr, F, FF, F, need[0] - 1, nullptr) == PC_ERR_SHAPE);
            CHECK(stub::launches.empty());
        }
    }
    stub::reset();
    CHECK(pc_cross_attention_backward(&a, F, F, F, F, FF, F, nullptr, nullptr, F, F, F, F, need[1], nullptr) == PC_OK);
    const int64_t dq = groups("k_attn_dq", cap), dkv = groups("k_attn_dkv", cap);
    CHECK((dq > 0) == (pairs > 0 && rows > 0));
    CHECK((dkv > 0) == (pairs > 0 && lk > 0));
    if (dkv) CHECK(dkv % (pairs * up(lk, 128)) == 0);
    // each launch in turn fails: the call stops there
    const size_t n = stub::launches.size();
    for (size_t i = 1; i <= n && i <= 4; ++i) {
        stub::reset();
        stub::fail_on_call = static_cast<int>(i);
        CHECK(pc_cross_attention_backward(&a, F, F, F, F, FF, F, nullptr, nullptr, F, F, F, F, need[1], nullptr) == PC_ERR_HIP);
        CHECK(stub::launches.size() == i);
    }
    stub::reset();
}

pc_norm_side side(int b, int l, int h, int d) {
    const pc_strides s = {int64_t(l) * h * d, int64_t(h) * d, d};
    pc_norm_side r;
    memset(&r, 0, sizeof r);
    r.batch = b;
    r.len = l;
    r.heads = h;
    r.x = r.y = F;
    r.dy = F;
    r.dx = F;
    r.dweight = FF;
    r.sx = r.sy = r.sdy = r.sdx = s;
    return r;
}

void norm(int dtype, int b, int l, int h, int d, int rot, uint64_t cap) {
    double f[64];
    for (int i = 0; i < 64; ++i) f[i] = (i % 2 ? -1.0 : 1.0) * 6.283185307179586 / (i + 1);
    const pc_norm_side q = side(b, l, h, d), k = side(2, 3, 1, d);
    for (int inter = 0; inter < 2; ++inter)
        for (int both = 0; both < 2; ++both) {
            int64_t need = -1;
            CHECK(pc_qk_norm_rope_workspace(&q, both ? &k : nullptr, dtype, d, rot, &need) == PC_OK && need >= 0);
            stub::reset();
            CHECK(pc_qk_norm_rope(&q, both ? &k : nullptr, dtype, d, rot, f, inter, 1e-6f, nullptr) == PC_OK);
            const int64_t tokens = int64_t(b) * l, g = groups("k_norm_rope", cap);
            CHECK(g <= tokens + 6 && (g > 0) == (tokens > 0 || both));
            for (const auto &x : stub::launches) CHECK(x.shm <= 32768);
            stub::reset();
            CHECK(pc_qk_norm_rope_backward(&q, both ? &k : nullptr, dtype, d, rot, f, inter, 1e-6f, F, need, nullptr) == PC_OK);
            const int64_t gb = groups("k_norm_rope", cap);
            CHECK(need == ((gb * d * 4 + 15) & ~int64_t(15)));
            CHECK(groups("k_norm_dw", cap) == 2 * up(d, 32));  // written also where no token is
            for (const auto &x : stub::launches) CHECK(x.shm <= 32768);
        }
    stub::reset();
    stub::fail_on_call = 1;
    const pc_norm_side one = side(1, 1, 1, d);
    CHECK(pc_qk_norm_rope(&one, nullptr, dtype, d, rot, f, 0, 1e-6f, nullptr) == PC_ERR_HIP);
    stub::reset();
}

}  // namespace

int main() {
    const uint64_t caps[] = {0, 1024};
    for (uint64_t c : caps) {
        CHECK(pc_set_max_dispatch_items(c) == PC_OK);
        const uint64_t cap = c ? c : 0xFFFFFFFFull;
        for (int dtype = 0; dtype < 3; ++dtype) {
            for (int d : {8, 32, 40, 64, 96, 128}) {
                attention(dtype, 1, 1, 1, 1, 1, 1, d, cap);
                attention(dtype, 1, 1, 1, 5000, 8, 2, d, cap);
                attention(dtype, 3, 7, 65, 129, 6, 3, d, cap);
                attention(dtype, 1, 40, 64, 70, 1, 1, d, cap);
                attention(dtype, 0, 4, 5, 6, 2, 1, d, cap);
                attention(dtype, 2, 0, 5, 6, 2, 1, d, cap);
                attention(dtype, 2, 3, 0, 6, 2, 2, d, cap);
                attention(dtype, 2, 3, 5, 0, 2, 2, d, cap);
                norm(dtype, 1, 1, 1, d, 0, cap);
                norm(dtype, 3, 17, 5, d, d / 16 * 16, cap);
                norm(dtype, 0, 17, 5, d, 0, cap);
                norm(dtype, 2, 3, 700, d, d / 16 * 16, cap);
                norm(dtype, 40, 64, 16, d, d / 16 * 16, cap);
            }
        }
    }
    CHECK(pc_set_max_dispatch_items(0) == PC_OK);
    const uint64_t cap = 0xFFFFFFFFull;
    attention(PC_BF16, 1, 1, 0x7FFFFFFF - 256, 4, 1, 1, 8, cap);   // most rows
    attention(PC_BF16, 1, 1, 1, 1 << 30, 1, 1, 8, cap);            // most keys
    attention(PC_F32, 1 << 14, 1, 64, 64, 64, 64, 128, cap);       // many pairs
    norm(PC_BF16, 1, 0x7FFFFFFF - 256, 1, 8, 0, cap);              // most tokens
    if (g_fails) {
        fprintf(stderr, "%d check(s) failed\n", g_fails);
        return 1;
    }
    printf("host checks passed\n");
    return 0;
}
