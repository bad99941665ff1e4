// The schedule that the tensor-core tile kernels share: barriers, tensor memory,
// the warp that issues the MMAs, and the output of a finished tile.
//
// A CTA is persistent, one per SM; a tile is two sub-tiles of 128 query rows against
// shared 128-key tiles of K and V, and a step of a sub-tile is S_t = Q_t K^T, the
// softmax warpgroup's P_t over S_t, and O_t += P_t V.  Tensor memory (512 columns x
// 128 lanes, fp32): S_0 [0,128), S_1 [128,256) (P_t in the first 64 columns of S_t),
// O_0 [256,256+D), O_1 [384,384+D).
#pragma once
#include "dev.cuh"

namespace pa {
namespace tiles {

using namespace dev;

__device__ __forceinline__ uint32_t col_s(int t) { return static_cast<uint32_t>(t) * 128u; }
__device__ __forceinline__ uint32_t col_o(int t) { return 256u + static_cast<uint32_t>(t) * 128u; }

// barrier indices.  K and V stages are released separately: a K stage as
// soon as the QK^T MMAs reading it finish, a V stage after the PV MMAs, so the
// next K tile is loaded while the current tile's softmax and PV still run.
// The CTA is persistent: rings, barriers and tensor memory carry over from one
// tile to the next, and the next tile's Q is loaded as soon as the current
// tile's last QK^T has read Q (QEMPTY), under the tile's last PV, softmax and
// epilogue.
enum : int {
    B_QFULL = 0,
    B_QEMPTY = 1,
    B_KFULL = 2,    // +stage (2)
    B_VFULL = 4,    // +stage (3)
    B_KEMPTY = 7,   // +stage (2)
    B_VEMPTY = 9,   // +stage (3)
    B_SFULL = 12,   // +sub-tile
    B_PFULL = 14,   // +sub-tile: keys 0..63 of P; +2: keys 64..127
    B_ODONE = 18,   // +sub-tile
    B_DRAIN = 20,
    B_SECOND = 21,  // split tiles: sub-tile 1's O, maximum and sum are there
    B_JOINED = 22,  // and have been read
    NUM_BARS = 23
};

// key tiles each sub-tile of a CTA tile needs (0 for an empty sub-tile)
struct TileShape {
    int n_sub[2];
    int n_tiles;
    bool split;   // key tile j belongs to sub-tile j % 2
    __device__ __forceinline__ int step(int i, int t) const { return split ? 2 * i + t : i; }   // i-th key tile of sub-tile t
};
template <bool SPLIT>
__device__ __forceinline__ TileShape tile_shape(const ExtendTile &tile, int tpt) {
    TileShape sh;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = t * tpt;
        if (first >= tile.n_tok) {
            sh.n_sub[t] = 0;
            continue;
        }
        const int last = min(tile.n_tok, first + tpt);   // one past the sub-tile's last token
        const int kend = tile.causal ? min(tile.key_end, tile.pos0 + last) : tile.key_end;
        sh.n_sub[t] = (kend - tile.key_begin + kTileKeys - 1) / kTileKeys;
    }
    sh.n_tiles = max(sh.n_sub[0], sh.n_sub[1]);
    sh.split = SPLIT && tile.split != 0 && sh.n_tiles >= 2;
    if (sh.split) {
        sh.n_sub[0] = (sh.n_tiles + 1) / 2;
        sh.n_sub[1] = sh.n_tiles / 2;
    }
    return sh;
}

// Hide the columns of an S row that a query does not see: from `lim` on, and
// [from, to) with a window.  A bit per column, so that a column costs little more
// than its select (two compares each: 4.7 us of the 71.4 that two chunks of 2048
// tokens take over a window of 1024).
template <bool WIN>
__device__ __forceinline__ void hide_columns(uint32_t (&sr)[128], int lim, int from, int to) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        auto below = [&](int n) { return n <= 32 * w ? 0u : n >= 32 * w + 32 ? ~0u : (1u << (n - 32 * w)) - 1u; };
        uint32_t seen = below(lim);
        if (WIN) seen &= ~(below(to) & ~below(from));
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (!(seen >> c & 1u)) sr[32 * w + c] = __float_as_uint(-INFINITY);
    }
}

// The warp that issues the MMAs, over the CTA's tiles.  C: the kernel's
// configuration (stages, tile bytes, instruction descriptors); q_s, k_s, v_s: its
// shared memory.  P comes in two halves, so that PV begins under the second half's
// exponentials.
template <int D, typename C, bool SPLIT>
__device__ __forceinline__ void issue_mmas(const ExtendParams &p, uint32_t bars, uint32_t q_s, uint32_t k_s, uint32_t v_s,
                                           uint32_t tmem, int tile_begin, int tile_end, int tpt, int lane, int *abort_flag) {
    auto bar = [&](int i) { return bars + 8u * i; };
    bool ok = true;
    const bool lead = lane == 0;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    // The warp runs the loop whole, on uniform conditions, and its leading
    // lane issues: descriptors stay in uniform registers (one lane alone
    // pays moves to them per MMA, and 2% more time).  The pipe takes the
    // next MMA only when the one before is nearly done, so whatever happens
    // between two MMAs beyond ~60 cycles leaves it idle: descriptors and
    // barrier addresses are running values, and barrier tests, a stage's
    // release and the next V tile's values sit in the gaps of the groups.
    const uint64_t q_desc[2] = {sdesc_sw128(q_s, 16, 1024), sdesc_sw128(q_s + C::QB, 16, 1024)};
    const uint64_t k_desc0 = sdesc_sw128(k_s, 16, 1024);
    const uint64_t v_desc0 = sdesc_sw128(v_s, C::HALF, 1024);
    const uint32_t sfull[2] = {bar(B_SFULL), bar(B_SFULL + 1)}, pfull[2] = {bar(B_PFULL), bar(B_PFULL + 1)};
    const uint32_t k_bar0 = bar(B_KFULL), v_bar0 = bar(B_VFULL);
    constexpr uint32_t kEmptyK = 8u * (B_KEMPTY - B_KFULL), kEmptyV = 8u * (B_VEMPTY - B_VFULL);
    uint32_t k_slot = 0, k_par = 0, v_slot = 0, v_par = 0;   // next K and V tile: ring slot, phase parity
    uint32_t k_bar = k_bar0, v_bar = v_bar0;                 // their full barriers
    uint64_t k_desc = k_desc0, v_desc = v_desc0;
    uint32_t p_par[2] = {0, 0};                              // parity of the next P
    uint32_t n_q = 0;
    // seen complete by a test in an MMA group
    bool p_ready[2] = {false, false}, p_rest = false, k_ready = false, v_ready = false;
    auto poll = [](bool &flag, uint32_t b, uint32_t parity) {
        if (!flag) flag = __all_sync(0xffffffffu, mbar_test_wait(b, parity));
    };
    auto need = [&](bool &flag, uint32_t b, uint32_t parity) -> bool {
        if (!flag && !warp_wait_spin(b, parity, abort_flag)) return false;
        flag = false;
        return true;
    };
    auto next_k = [&] {
        const bool wrap = k_slot + 1 == C::NSK;
        k_slot = wrap ? 0 : k_slot + 1;
        k_par ^= wrap ? 1u : 0u;
        k_bar = k_bar0 + 8u * k_slot;
        k_desc = sdesc_advance(k_desc0, k_slot * C::KVB);
    };
    auto next_v = [&] {
        const bool wrap = v_slot + 1 == C::NSV;
        v_slot = wrap ? 0 : v_slot + 1;
        v_par ^= wrap ? 1u : 0u;
        v_bar = v_bar0 + 8u * v_slot;
        v_desc = sdesc_advance(v_desc0, v_slot * C::KVB);
    };
    // MMA groups; gap(kk) runs behind MMA kk
    auto qk = [&](int t, auto gap) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk / 4) * C::HALF + (kk % 4) * 32;
            tc_mma_if(lead, tm + col_s(t), sdesc_advance(q_desc[t], off), sdesc_advance(k_desc, off),
                      C::IDESC_QK, kk > 0 ? 1u : 0u);
            gap(kk);
        }
        tc_commit_if(lead, sfull[t]);
    };
    // (the first half of P has been waited for)
    auto pv = [&](int t, uint32_t accumulate, auto gap) -> bool {
#pragma unroll
        for (int kk = 0; kk < kTileKeys / 16; ++kk) {
            if (kk == 3) poll(p_rest, pfull[t] + 16, p_par[t]);
            if (kk == kTileKeys / 32) {
                if (!need(p_rest, pfull[t] + 16, p_par[t])) return false;
                tc_fence_after();
                p_par[t] ^= 1u;
            }
            tc_mma_ts_if(lead, tm + col_o(t), tm + col_s(t) + kk * 8, sdesc_advance(v_desc, kk * 2048),
                         C::IDESC_PV, kk > 0 ? 1u : accumulate);
            gap(kk);
        }
        return true;
    };
    auto nothing = [](int) {};
    const int ti_end = __shfl_sync(0xffffffffu, tile_end, 0);
    for (int ti = __shfl_sync(0xffffffffu, tile_begin, 0); ti < ti_end && ok; ++ti) {
        const ExtendTile tile = p.tiles[p.cta_tiles[ti]];
        const TileShape sh = tile_shape<SPLIT>(tile, tpt);
        const int n0 = __shfl_sync(0xffffffffu, sh.n_sub[0], 0), n1 = __shfl_sync(0xffffffffu, sh.n_sub[1], 0);
        const int n = max(n0, n1), n_both = min(n0, n1);
        ok = warp_wait_spin(bar(B_QFULL), n_q & 1, abort_flag);
        ++n_q;
        if (!ok || n == 0) {
            if (ok) tc_commit_if(lead, bar(B_QEMPTY));
            continue;
        }
        if (SPLIT && __shfl_sync(0xffffffffu, sh.split ? 1 : 0, 0)) {
            // a key tile for one sub-tile, the next for the other
            auto next_qk = [&](int t, bool last) -> bool {
                if (!need(k_ready, k_bar, k_par)) return false;
                tc_fence_after();
                qk(t, nothing);
                tc_commit_if(lead, k_bar + kEmptyK);
                next_k();
                if (last) tc_commit_if(lead, bar(B_QEMPTY));
                return true;
            };
            ok = next_qk(0, false) && next_qk(1, n0 + n1 == 2);
            for (int i = 0; i < n0 && ok; ++i) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int nt = t ? n1 : n0;
                    if (!ok || i >= nt) continue;
                    ok = need(v_ready, v_bar, v_par) && need(p_ready[t], pfull[t], p_par[t]);
                    if (!ok) break;
                    tc_fence_after();
                    ok = pv(t, i > 0 ? 1u : 0u, nothing);
                    if (!ok) break;
                    tc_commit_if(lead, v_bar + kEmptyV);
                    next_v();
                    if (i + 1 < nt) ok = next_qk(t, 2 * (i + 1) + t + 1 == n0 + n1);
                    else tc_commit_if(lead, bar(B_ODONE + t));
                }
            }
            continue;
        }
        if (!need(k_ready, k_bar, k_par)) { ok = false; break; }
        tc_fence_after();
        if (n0 > 0) qk(0, nothing);
        if (n1 > 0) qk(1, nothing);
        tc_commit_if(lead, k_bar + kEmptyK);   // K tile 0 read by both QK^T
        if (n == 1) tc_commit_if(lead, bar(B_QEMPTY));
        next_k();
        int j = 0;
        // steps whose two sub-tiles both go on: PV_0(j) QK_0(j+1) PV_1(j)
        // QK_1(j+1)
        for (; j + 1 < n_both; ++j) {
            if (!need(v_ready, v_bar, v_par) || !need(p_ready[0], pfull[0], p_par[0])) { ok = false; break; }
            tc_fence_after();
            ok = pv(0, j > 0 ? 1u : 0u, [&](int kk) {
                if (kk == 5) poll(k_ready, k_bar, k_par);
            });
            if (!ok || !need(k_ready, k_bar, k_par)) { ok = false; break; }
            tc_fence_after();
            // overwrites S_0: issued after the PV that reads P_0
            qk(0, [&](int kk) {
                if (kk == D / 16 - 3) poll(p_ready[1], pfull[1], p_par[1]);
            });
            if (!need(p_ready[1], pfull[1], p_par[1])) { ok = false; break; }
            tc_fence_after();
            ok = pv(1, j > 0 ? 1u : 0u, nothing);
            if (!ok) break;
            qk(1, [&](int kk) {
                if (kk == 0) tc_commit_if(lead, v_bar + kEmptyV);   // V tile j read by both PV
                if (kk == 1) next_v();
                if (kk == 2) poll(v_ready, v_bar, v_par);
                if (kk == D / 16 - 2) poll(p_ready[0], pfull[0], p_par[0]);
            });
            tc_commit_if(lead, k_bar + kEmptyK);   // K tile j+1 read by both QK^T
            next_k();
        }
        if (ok && j > 0 && j + 1 == n) tc_commit_if(lead, bar(B_QEMPTY));
        // the last steps, of one sub-tile or without a QK^T
        for (; j < n && ok; ++j) {
            ok = need(v_ready, v_bar, v_par);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int nt = t ? n1 : n0;
                if (!ok || j >= nt) continue;
                ok = need(p_ready[t], pfull[t], p_par[t]);
                if (!ok) break;
                tc_fence_after();
                ok = pv(t, j > 0 ? 1u : 0u, nothing);
                if (!ok) break;
                if (j + 1 < nt) {
                    if (!k_ready) ok = warp_wait_spin(k_bar, k_par, abort_flag);
                    if (!ok) break;
                    k_ready = true;
                    tc_fence_after();
                    qk(t, nothing);
                } else {
                    tc_commit_if(lead, bar(B_ODONE + t));
                }
            }
            if (!ok) break;
            tc_commit_if(lead, v_bar + kEmptyV);
            next_v();
            if (j + 1 < n) {
                tc_commit_if(lead, k_bar + kEmptyK);
                next_k();
                k_ready = false;
                if (j + 2 == n) tc_commit_if(lead, bar(B_QEMPTY));
            }
        }
    }
    if (!ok && lead) raise_abort(abort_flag, p.err, kErrTimeout);
    // every MMA of this CTA must finish before tensor memory is released
    tc_commit_if(lead, bar(B_DRAIN));
    if (!mbar_wait(bar(B_DRAIN), 0, nullptr) && lead) atomicOr(p.err, kErrTimeout);
    __syncwarp();
}

// N columns of a row's O (tensor memory at o_at, this warp's lanes) times `inv`; with a
// second sub-tile's O at `other`, that one times `inv2` added.
template <int N>
__device__ __forceinline__ void load_output(uint32_t (&x)[N], uint32_t o_at, uint32_t other, bool two, float inv, float inv2) {
#pragma unroll
    for (int c = 0; c < N; c += 32) tmem_ld32(o_at + c, *reinterpret_cast<uint32_t(*)[32]>(&x[c]));
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * inv);
    if (two) {
#pragma unroll
        for (int c = 0; c < N; c += 32) {
            uint32_t y[32];
            tmem_ld32(other + c, y);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
                x[c + e] = __float_as_uint(fmaf(__uint_as_float(y[e]), inv2, __uint_as_float(x[c + e])));
        }
    }
}

// A row's output of a finished tile: O times `inv` (and the second sub-tile's), as bf16
// into its row of out, or as fp32 into its partial.  read() runs once O has been read.
template <int D, typename Read>
__device__ __forceinline__ void store_output(const ExtendParams &p, uint32_t o_at, uint32_t other, bool two, bool tok_valid,
                                             int part, int tok, int h, int64_t slot, float inv, float inv2, int lane, Read read) {
    if (part < 0) {
        // Four neighbouring lanes hold four rows; their 32-byte pieces are
        // exchanged so that a store writes 128 consecutive bytes of 8 rows
        // (a piece of 32 rows each: 80 cycles a store, 5000 an epilogue,
        // with the MMA thread's requests queued behind them).
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        const int64_t mine = tok_valid ? (static_cast<int64_t>(tok) * p.num_heads_q + h) * D : -1;
        int64_t at[4];   // rows of the four lanes
#pragma unroll
        for (int s = 0; s < 4; ++s) at[s] = __shfl_sync(0xffffffffu, mine, (lane & ~3) + s);
#pragma unroll 1
        for (int c = 0; c < D; c += 64) {
            uint32_t orr[64], w[32];
            load_output<64>(orr, o_at + c, other + c, two, inv, inv2);
            if (c + 64 >= D) read();
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = pack_bf16x2(__uint_as_float(orr[2 * e]), __uint_as_float(orr[2 * e + 1]));
#pragma unroll
            for (int bit = 1; bit <= 2; bit *= 2) {
                const bool up = lane & bit;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k & bit) continue;   // pieces k and k + bit
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint32_t &lo = w[8 * k + e], &hi = w[8 * (k + bit) + e];
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
                        if (up) lo = got;
                        else hi = got;
                    }
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (at[s] >= 0)
                    st_row_v8(wide, p.out + at[s] + c + 16 * (lane & 3), w[8 * s], w[8 * s + 1], w[8 * s + 2],
                              w[8 * s + 3], w[8 * s + 4], w[8 * s + 5], w[8 * s + 6], w[8 * s + 7]);
        }
    } else {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t orr[32];
            load_output<32>(orr, o_at + c, other + c, two, inv, inv2);
            if (c + 32 >= D) read();
            if (!tok_valid) continue;
            float *dst = p.o_part + (slot * p.num_heads_q + h) * D + c;
#pragma unroll
            for (int q8 = 0; q8 < 4; ++q8)
                st_global_v8(dst + q8 * 8, orr[q8 * 8 + 0], orr[q8 * 8 + 1], orr[q8 * 8 + 2], orr[q8 * 8 + 3],
                             orr[q8 * 8 + 4], orr[q8 * 8 + 5], orr[q8 * 8 + 6], orr[q8 * 8 + 7]);
        }
    }
}

// The joint result of a split tile's sub-tiles, for the warpgroup of sub-tile 0: m and l
// become those of all keys, and a0, a1 what each sub-tile's O counts in it.
struct Joined {
    float a0 = 1.f, a1 = 0.f;
    __device__ __forceinline__ void join(float &m, float &l, float2 second) {
        const float top = fmaxf(m, second.x);
        a0 = m == -INFINITY ? 0.f : ex2(m - top);
        a1 = second.x == -INFINITY ? 0.f : ex2(second.x - top);
        m = top;
        l = l * a0 + second.y * a1;
    }
};

}  // namespace tiles
}  // namespace pa
