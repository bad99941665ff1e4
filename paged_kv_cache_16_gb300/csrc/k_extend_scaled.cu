// Extend / chunked-prefill and shared-prefix attention on the tensor cores over
// block-scaled 8-bit caches: the schedule of k_extend.cu (two 128-row sub-tiles
// per CTA tile against shared 128-key tiles; TMA producer, one MMA-issuing thread,
// a softmax warpgroup per sub-tile, accumulators in tensor memory), with the codes
// themselves as operands.  K and V tiles are 16-bit copies of the codes, exact: K
// in bf16 beside the bf16 queries, V in f16 beside f16 weights.  The scales enter
// in fp32, per block of 16 key columns, as in the split-KV kernel:
//   w = 2^(s + log2 vs - R), s = softmax_scale log2(e) ks <q, kcode>,
//   O += w vcode,  L += (sum of the block's w) / vs,  out = O / L,
// so a tile loses nothing to the quantisation's form (bf16 weights and dequantised
// bf16 K and V gave 2.6 times the error of the output's own rounding; this adds
// nothing visible).  Three factors per (block, kv head), written by the expansion
// kernel as one 16-byte record, travel with the V stage, which is not given back
// before its weights have been used: a softmax warp waits for it under QK^T.
//
// Two chunks of 2048 tokens over 2304 and 4864 (Hq 32, Hkv 8, D 128): 204 us at
// 2070 MHz, 1516 TFLOP/s, where the kernel of the E4M3 caches with one scale takes
// 244.  A step of 128 keys has 2048 cycles of MMAs and takes ~2800 (tensor pipe
// active 68%, issue 43%): what the MMA warp does between two MMAs, and the chain
// S -> softmax -> P of a sub-tile (~1500 cycles), which its own PV and QK^T follow.
// P is handed over in halves, so that PV begins under the second half's
// exponentials (3%; after a quarter or three quarters 1% more than that), by one
// arrival per warp (1.5%).  Between two tiles go ~3 steps' time: the last softmax,
// the epilogue and the first QK^T in a row.  Measured and not kept, as parts of the
// time then: ring indices by division and all commits at the groups' ends +8%;
// weights through shared memory, QK^T a step ahead, +23% (every operand from shared
// memory fills its bandwidth); one S buffer for both sub-tiles and QK^T a step
// ahead, +39% with one MMA thread, +11% with one for QK^T and one for PV; an MMA
// thread per sub-tile, +25%, taking turns at the pipe +2%; two threads per row +15%;
// the first half's weights against the old reference, checked by their sum, beside
// the second half's maximum, S read again where a row needs a new one, +3%; the
// blocks' factors read from shared memory where they are used instead of held, +2%;
// the next tile's first QK^T in a tile's last step +2%, one loop body for full and
// last steps +23%; stages given back by a softmax warp, tile descriptions in shared
// memory, three K and two V stages: no change.
#include "dev.cuh"

namespace pa {
namespace {

using namespace dev;

template <int D>
struct ScaledExtCfg {
    static constexpr int NH = D / 64;
    static constexpr int HALF = 128 * 128;            // [128 rows][64] bf16 half tile
    static constexpr int QB = NH * HALF;              // one Q sub-tile
    static constexpr int KVB = NH * HALF;             // K (or V) tile bytes per stage
    static constexpr int NSK = 2;                     // K stages
    static constexpr int NSV = 3;                     // V stages (V waits longest for its stage)
    static constexpr int THREADS = 384;               // 3 warpgroups
    // registers per thread after the split (launch: 168 x 384 = 64512):
    // 120 x 128 for the load / MMA warpgroup + 192 x 256 for the two softmax
    // warpgroups = 64512
    static constexpr int REGS_CTRL = 120;
    static constexpr int REGS_SOFTMAX = 192;
    static_assert(REGS_CTRL * 128 + REGS_SOFTMAX * 256 <= 168 * 384, "register split exceeds the launch");
    static constexpr int FACTORS = NSV * (kTileKeys / kBlockSize) * 16;   // a record per block of a V stage
    static constexpr int TILE_SMEM = 2 * QB + (NSK + NSV) * KVB + FACTORS;
    // one CTA per SM: it owns all 512 tensor-memory columns
    static constexpr int SMEM = (TILE_SMEM + 2048 < 120 * 1024) ? 120 * 1024 : TILE_SMEM + 2048;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t IDESC_QK = idesc_bf16(128, 128, false, false);
    static constexpr uint32_t IDESC_PV = idesc_bf16(128, D, false, true) & ~((1u << 7) | (1u << 10));   // f16 A and B
};


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
    NUM_BARS = 21
};

// key tiles each sub-tile of a CTA tile needs (0 for an empty sub-tile)
struct TileShape {
    int n_sub[2];
    int n_tiles;
};
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
    return sh;
}

template <int D>
__global__ void __launch_bounds__(384, 1)
scaled_extend_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const ScaledExtendParams sp) {
    using C = ScaledExtCfg<D>;
    const ExtendParams &p = sp.base;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    __shared__ uint32_t tmem_base_slot;
    __shared__ __align__(8) uint64_t bars[NUM_BARS];

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    auto q_s = [&](int t) { return base + static_cast<uint32_t>(t) * C::QB; };
    auto k_s = [&](int s) { return base + 2 * C::QB + static_cast<uint32_t>(s) * C::KVB; };
    auto v_s = [&](int s) { return base + 2 * C::QB + static_cast<uint32_t>(C::NSK + s) * C::KVB; };
    // factors of block `page` of V stage s: {ks * scale, log2 vs, 1 / vs, unused}
    auto f_s = [&](int s, int page) {
        return base + 2 * C::QB + static_cast<uint32_t>(C::NSK + C::NSV) * C::KVB + 16u * (8 * s + page);
    };
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    grid_launch_dependents();
    grid_dep_wait();    // the work list and caches come from earlier kernels of the stream
    // this CTA's tiles, longest first (the planner's greedy assignment)
    const int tile_begin = p.cta_tile_begin[blockIdx.x];
    const int tile_end = p.cta_tile_begin[blockIdx.x + 1];
    if (tile_begin >= tile_end) return;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // (uniform to the compiler)
    const int lane = threadIdx.x & 31;
    const int G = p.group;
    const int tpt = kTileRows / G;                    // tokens per 128-row sub-tile

    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(bar(B_QFULL), 1);
        mbar_init(bar(B_QEMPTY), 1);
        for (int s = 0; s < C::NSK; ++s) {
            mbar_init(bar(B_KFULL + s), 1);
            mbar_init(bar(B_KEMPTY + s), 1);
        }
        for (int s = 0; s < C::NSV; ++s) {
            mbar_init(bar(B_VFULL + s), 1);
            mbar_init(bar(B_VEMPTY + s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(B_SFULL + t), 1);
            mbar_init(bar(B_PFULL + t), 4);       // a warp each
            mbar_init(bar(B_PFULL + 2 + t), 4);
            mbar_init(bar(B_ODONE + t), 1);
        }
        mbar_init(bar(B_DRAIN), 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_base_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_slot;
    if (warp < 4) {
      // warpgroup 0: loads and MMA issue, with few registers
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CTRL));
      if (warp == 0) {
        // -------------------------------------------------------- producer --
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
        int issued[2] = {0, 0};   // K and V tiles whose loads were issued (over all tiles)
        int n_q_loads = 0;
        bool ok = true;
        for (int ti = tile_begin; ti < tile_end && ok; ++ti) {
            const ExtendTile tile = p.tiles[p.cta_tiles[ti]];
            const TileShape sh = tile_shape(tile, tpt);
            // Q of this tile, once the previous tile's QK^T no longer read Q
            if (n_q_loads > 0 && !warp_wait(bar(B_QEMPTY), (n_q_loads - 1) & 1, &abort_flag)) {
                if (lane == 0) raise_abort(&abort_flag, p.err, kErrTimeout);
                break;
            }
            const int n_q = sh.n_sub[1] > 0 ? 2 : 1;
            // each box is tpt tokens x G heads x 64 dims: tpt * G rows of
            // 128 bytes (128 rows unless G does not divide 128)
            if (lane == 0) mbar_arrive_expect_tx(bar(B_QFULL), n_q * C::NH * tpt * G * 128);
            __syncwarp();
            if (lane < n_q * C::NH) {
                const int t = lane / C::NH, half = lane % C::NH;
                tma_load_3d(q_s(t) + half * C::HALF, &tm_q, half * 64, tile.kv_head * G, tile.t0 + t * tpt,
                            bar(B_QFULL));
            }
            ++n_q_loads;
            // the copies of a request's blocks are consecutive, so a key tile is
            // 128 consecutive rows of them: one box per 64 columns of K and of V
            // (16 boxes of one block each and 8 bulk copies of single records cost
            // the producer 8% of the kernel's time).  Rows behind the key range
            // belong to other requests or to none: masked columns, and value
            // rows that the softmax warps zero
            const int32_t dst0 = p.block_table[static_cast<int64_t>(tile.req) * p.max_blocks + tile.key_begin / kBlockSize];
            const int pg_end = (tile.key_end - tile.key_begin + kBlockSize - 1) / kBlockSize;
            if (dst0 < 0 || dst0 + pg_end > p.num_blocks) {   // (not from the planner)
                if (lane == 0) raise_abort(&abort_flag, p.err, kErrBlockRange);
                break;
            }
            for (int j = 0; j < sh.n_tiles; ++j) {
                const int pg0 = j * (kTileKeys / kBlockSize);
                const int pages = min(kTileKeys / kBlockSize, pg_end - pg0);
#pragma unroll
                for (int tensor = 0; tensor < 2; ++tensor) {
                    const int ns = tensor ? C::NSV : C::NSK;
                    const int s = issued[tensor] % ns, n = issued[tensor] / ns;
                    const int empty = tensor ? B_VEMPTY : B_KEMPTY;
                    const int full = tensor ? B_VFULL : B_KFULL;
                    if (n > 0 && !warp_wait(bar(empty + s), (n & 1) ^ 1, &abort_flag)) {
                        if (lane == 0) raise_abort(&abort_flag, p.err, kErrTimeout);
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(bar(full + s), C::KVB + (tensor ? 16u * pages : 0u));
                    __syncwarp();
                    if (lane < C::NH)
                        tma_load_3d((tensor ? v_s(s) : k_s(s)) + lane * C::HALF, tensor ? &tm_v : &tm_k, lane * 64,
                                    tile.kv_head, (dst0 + pg0) * kBlockSize, bar(full + s));
                    else if (tensor && lane == C::NH)
                        bulk_load(f_s(s, 0), sp.factors + static_cast<int64_t>(tile.kv_head) * p.num_blocks + dst0 + pg0,
                                  16u * pages, bar(full + s));
                    ++issued[tensor];
                }
                if (!ok) break;
            }
        }
        if (lane == 0) {
            // no TMA write may outlive the CTA
            if (n_q_loads > 0 && !mbar_wait(bar(B_QFULL), (n_q_loads - 1) & 1, nullptr)) atomicOr(p.err, kErrTimeout);
            for (int tensor = 0; tensor < 2; ++tensor) {
                const int ns = tensor ? C::NSV : C::NSK;
                for (int k = issued[tensor] - 1; k >= 0 && k >= issued[tensor] - ns; --k) {
                    const int s = k % ns, n = k / ns;
                    if (!mbar_wait(bar((tensor ? B_VFULL : B_KFULL) + s), n & 1, nullptr))
                        atomicOr(p.err, kErrTimeout);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer --
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
        const uint64_t q_desc[2] = {sdesc_sw128(q_s(0), 16, 1024), sdesc_sw128(q_s(1), 16, 1024)};
        const uint64_t k_desc0 = sdesc_sw128(k_s(0), 16, 1024);
        const uint64_t v_desc0 = sdesc_sw128(v_s(0), C::HALF, 1024);
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
            if (!flag && !warp_wait_spin(b, parity, &abort_flag)) return false;
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
            const TileShape sh = tile_shape(tile, tpt);
            const int n0 = __shfl_sync(0xffffffffu, sh.n_sub[0], 0), n1 = __shfl_sync(0xffffffffu, sh.n_sub[1], 0);
            const int n = max(n0, n1), n_both = min(n0, n1);
            ok = warp_wait_spin(bar(B_QFULL), n_q & 1, &abort_flag);
            ++n_q;
            if (!ok || n == 0) {
                if (ok) tc_commit_if(lead, bar(B_QEMPTY));
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
                        if (!k_ready) ok = warp_wait_spin(k_bar, k_par, &abort_flag);
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
        if (!ok && lead) raise_abort(&abort_flag, p.err, kErrTimeout);
        // every MMA of this CTA must finish before tensor memory is released
        tc_commit_if(lead, bar(B_DRAIN));
        if (!mbar_wait(bar(B_DRAIN), 0, nullptr) && lead) atomicOr(p.err, kErrTimeout);
        __syncwarp();
      }
    } else {
        // ------------------------------------------- softmax + epilogue --
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
        const int t = (warp - 4) / 4;            // sub-tile of this warpgroup
        const int quarter = warp & 3;            // tensor-memory lanes 32*quarter .. +31
        const int row = quarter * 32 + lane;
        const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        int scnt = 0, ocnt = 0;                  // S tiles and outputs consumed by this sub-tile
        int vbase = 0;                           // V tiles of the previous tiles of this CTA
        int v_seen = 0;                          // one past the last V tile waited for
        bool ok = true;
        for (int ti = tile_begin; ti < tile_end && ok; ++ti) {
            const ExtendTile tile = p.tiles[p.cta_tiles[ti]];
            const TileShape sh = tile_shape(tile, tpt);
            const int i = t * tpt + row / G;         // token of this row within the tile
            const int gq = row % G;
            // rows past tpt * G (when G does not divide 128) are padding
            const bool tok_valid = row < tpt * G && i < tile.n_tok;
            const int pos_lim = tile.causal ? tile.pos0 + i + 1 : 0x7fffffff;  // keys < pos_lim
            const int row_end = min(tile.key_end, pos_lim);
            const int n_mine = t ? sh.n_sub[1] : sh.n_sub[0];
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n_mine; ++j) {
                const int kt0 = tile.key_begin + j * kTileKeys;
                // Behind tiles whose empty second sub-tile passed this warpgroup by,
                // S comes first: the parity of a V barrier tells two neighbouring
                // phases apart only, and this warpgroup has not seen the phase
                // before the one asked for.  S completes behind every MMA of the
                // tiles before, so that phase is over.  (S first in every tile:
                // 214.0 us instead of 212.8 for the two chunks above.)
                const bool s_first = vbase + j >= v_seen + C::NSV;
                if (s_first && !warp_wait(bar(B_SFULL + t), scnt & 1, &abort_flag)) { ok = false; break; }
                v_seen = vbase + j + 1;
                // the factors of the tile's blocks, which came with its V stage,
                // while S is being computed; blocks past the key range have none,
                // and masked columns
                const int vs_stage = (vbase + j) % C::NSV;
                if (!warp_wait(bar(B_VFULL + vs_stage), ((vbase + j) / C::NSV) & 1, &abort_flag)) { ok = false; break; }
                float fs[8], lv[8], iv[8];
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const uint4 f = lds_v4(f_s(vs_stage, b));
                    fs[b] = __uint_as_float(f.x);
                    lv[b] = __uint_as_float(f.y);
                    iv[b] = __uint_as_float(f.z);
                }
                if (tile.key_end - kt0 < kTileKeys) {
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        if (kt0 + kBlockSize * b >= tile.key_end) { fs[b] = 1.f; lv[b] = 0.f; iv[b] = 0.f; }
                }
                if (!s_first && !warp_wait(bar(B_SFULL + t), scnt & 1, &abort_flag)) { ok = false; break; }
                ++scnt;
                tc_fence_after();
                const int lim = row_end - kt0;       // columns < lim are visible
                // the whole S row in registers: four loads, one wait
                uint32_t sr[128];
                tmem_ld32(t_row + col_s(t) + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
                tmem_ld32(t_row + col_s(t) + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
                tmem_ld32(t_row + col_s(t) + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
                tmem_ld32(t_row + col_s(t) + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
                tmem_wait_ld();
                if (lim < kTileKeys) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c >= lim) sr[c] = __float_as_uint(-INFINITY);
#pragma unroll
                    for (int b = 0; b < 8; ++b)   // none of the block: its scale, NaN even, plays no part
                        if (kBlockSize * b >= lim) fs[b] = 1.f;
                }
                // row max of s + log2 vs
                float mxs = -INFINITY;
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    auto s = [&](int c) { return __uint_as_float(sr[16 * b + c]); };
                    float mx0 = max3(s(0), s(1), s(2)), mx1 = max3(s(3), s(4), s(5));
                    mx0 = max3(mx0, s(6), s(7));
                    mx1 = max3(mx1, s(8), s(9));
                    mx0 = max3(mx0, s(10), s(11));
                    mx1 = max3(mx1, s(12), s(13));
                    mx0 = max3(mx0, s(14), s(15));
                    mxs = fmaxf(mxs, fmaf(fmaxf(mx0, mx1), fs[b], lv[b]));
                }
                const bool need = mxs > m + 8.f;
                float alpha = 1.f;
                if (need) {
                    alpha = ex2(m - mxs);
                    m = mxs;
                    l *= alpha;
                }
                const float nref = m == -INFINITY ? 0.f : -m;
                // w = exp2(s + log2 vs - m) as f16 pairs, packed in place (entry e
                // takes columns 2e and 2e+1, which are read before entry e is
                // written), then stored over the first 64 columns of S; the
                // scale-and-shift and the sums run on packed fp32 pairs
                uint64_t l2 = f32x2(0.f, 0.f);
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const uint64_t scale2 = f32x2(fs[b], fs[b]), shift2 = f32x2(lv[b] + nref, lv[b] + nref);
                    uint64_t w[2];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int c = 16 * b + 2 * e;
                        float x0, x1;
                        f32x2_split(fma_f32x2(f32x2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), scale2, shift2),
                                    x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        w[e & 1] = e < 2 ? f32x2(p0, p1) : add_f32x2(w[e & 1], f32x2(p0, p1));
                        sr[8 * b + e] = pack_f16x2(p0, p1);
                    }
                    l2 = fma_f32x2(add_f32x2(w[0], w[1]), f32x2(iv[b], iv[b]), l2);
                    if (b == 3) {   // the first half of P, under which its PV can begin
                        tmem_st32(t_row + col_s(t) + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
                        if (j >= 1 && __any_sync(0xffffffffu, need)) {
                            // O_t holds the tiles before j (their PV completed before S_t(j) did)
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t orr[32];
                                tmem_ld32(t_row + col_o(t) + c, orr);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
                                tmem_st32(t_row + col_o(t) + c, orr);
                            }
                        }
                        tmem_wait_st();
                        // value rows past the end of the key range may hold anything
                        // (unwritten slots, stale blocks, NaN): zero them so that
                        // 0 * row stays 0 inside the MMA.  Each sub-tile that reads
                        // the last V tile zeroes them before handing over its P, so
                        // the PV after it sees zeros (both write the same zeros).
                        const int valid_keys = tile.key_end - kt0;
                        if (valid_keys < kTileKeys && j == sh.n_tiles - 1) {
                            const int s = vs_stage;   // (landed: waited for above)
                            if (row >= valid_keys) {
#pragma unroll
                                for (int h = 0; h < C::NH; ++h)
#pragma unroll
                                    for (int ch = 0; ch < 8; ++ch) {
                                        const uint32_t a = v_s(s) + h * C::HALF + row * 128 + ch * 16;
                                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
                                    }
                            }
                            fence_proxy_async_smem();
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(B_PFULL + t));
                    }
                }
                float l0, l1;
                f32x2_split(l2, l0, l1);
                l += l0 + l1;
                tmem_st32(t_row + col_s(t) + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_PFULL + 2 + t));
            }
            if (!ok) break;
            vbase += sh.n_tiles;
            // ------------------------------------------------- epilogue --
            if (n_mine == 0) continue;
            if (!warp_wait(bar(B_ODONE + t), ocnt & 1, &abort_flag)) { ok = false; break; }
            ++ocnt;
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : 1.f / l;   // no visible key: 0; a NaN stays one
            const int tok = tile.t0 + i;
            const int h = tile.kv_head * G + gq;
            int64_t slot = -1;
            if (tile.part >= 0 && tok_valid)
                slot = static_cast<int64_t>(p.part_offset[tok * p.n_groups + tile.kv_head / p.heads_per_group]) +
                       tile.part;
            if (tile.part < 0) {
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
                    tmem_ld32(t_row + col_o(t) + c, *reinterpret_cast<uint32_t(*)[32]>(&orr[0]));
                    tmem_ld32(t_row + col_o(t) + c + 32, *reinterpret_cast<uint32_t(*)[32]>(&orr[32]));
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        w[e] = pack_bf16x2(__uint_as_float(orr[2 * e]) * inv, __uint_as_float(orr[2 * e + 1]) * inv);
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
                    tmem_ld32(t_row + col_o(t) + c, orr);
                    tmem_wait_ld();
                    if (!tok_valid) continue;
                    float *dst = p.o_part + (slot * p.num_heads_q + h) * D + c;
#pragma unroll
                    for (int q8 = 0; q8 < 4; ++q8)
                        st_global_v8(dst + q8 * 8, __float_as_uint(__uint_as_float(orr[q8 * 8 + 0]) * inv),
                                     __float_as_uint(__uint_as_float(orr[q8 * 8 + 1]) * inv),
                                     __float_as_uint(__uint_as_float(orr[q8 * 8 + 2]) * inv),
                                     __float_as_uint(__uint_as_float(orr[q8 * 8 + 3]) * inv),
                                     __float_as_uint(__uint_as_float(orr[q8 * 8 + 4]) * inv),
                                     __float_as_uint(__uint_as_float(orr[q8 * 8 + 5]) * inv),
                                     __float_as_uint(__uint_as_float(orr[q8 * 8 + 6]) * inv),
                                     __float_as_uint(__uint_as_float(orr[q8 * 8 + 7]) * inv));
                }
            }
            // the partial's weight 2^m l in the merge, kept as l = 1 (L holds the
            // range of 1 / vs); a NaN takes the merge over
            if (tok_valid && tile.part >= 0)
                p.ml_part[slot * p.num_heads_q + h] =
                    l == 0.f ? make_float2(-INFINITY, 0.f) : make_float2(l != l ? 3.0e38f : m + lg2(l), 1.f);
            tc_fence_before();
        }
        if (!ok) raise_abort(&abort_flag, p.err, kErrTimeout);
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int D>
cudaError_t configure() {
    // the attribute is per function and device; setting it again is harmless
    return cudaFuncSetAttribute(scaled_extend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, ScaledExtCfg<D>::SMEM);
}

template <int D>
cudaError_t launch_t(int grid, const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                     const ScaledExtendParams &p, cudaStream_t stream, bool pdl) {
    using C = ScaledExtCfg<D>;
    return launch_ex(scaled_extend_kernel<D>, dim3(grid), dim3(C::THREADS), C::SMEM, stream, pdl, tm_q, tm_k, tm_v, p);
}

}  // namespace

cudaError_t prepare_scaled_extend(int head_dim) {
    if (head_dim == 128) return configure<128>();
    if (head_dim == 64) return configure<64>();
    return cudaErrorInvalidValue;
}

cudaError_t launch_scaled_extend(int head_dim, int grid, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                          const CUtensorMap &tm_v, const ScaledExtendParams &p, cudaStream_t stream, bool pdl) {
    if (grid <= 0) return cudaSuccess;
    if (head_dim == 128) return launch_t<128>(grid, tm_q, tm_k, tm_v, p, stream, pdl);
    if (head_dim == 64) return launch_t<64>(grid, tm_q, tm_k, tm_v, p, stream, pdl);
    return cudaErrorInvalidValue;
}

}  // namespace pa
