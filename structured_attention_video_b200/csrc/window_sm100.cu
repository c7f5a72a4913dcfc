// window_sm100.cu -- window attention forward on the sm_100a tensor cores (bfloat16
// inputs, float32 sums and softmax, the probabilities rounded to bfloat16 as
// operands of the second product).
//
// Persistent, 512 threads a CTA, one CTA an SM.  A problem is one head and a pair of
// 128-row query tiles; its keys are the two runs of 64-key blocks that some row of the
// pair sees, two blocks a chunk.  Either each CTA takes whole problems (the longest
// first), or, where those would leave SMs idle, the chunks of all problems form one line
// that the CTAs divide evenly: a problem cut by a boundary leaves its parts' unscaled sums,
// maxima and row sums in the workspace, and a second kernel joins them in order.  Roles:
// warp 12 loads keys, warp 14 queries and values (TMA), warps 13 and 15 issue the products
// of tile 0 and 1, warps 0-3 and 4-7 are the softmax of tile 0 and 1 (one query row a
// thread), warps 8-11 the epilogue.  Keys go in halves of 64: each tile has two S buffers
// of 64 columns in tensor memory, so the logits of the next half are ready while the
// softmax works on this one; P overwrites S in place.  The running maximum moves only
// when it grows by more than 2^8, so O is rarely rescaled.
//
// Bound by the exponentials (16 a clock and SM, 2 tiles x 128 x 64 a half) together with
// the issue slots of the softmax warps, then by the products.  A 480p chunk of 4680
// queries that see 18720 keys, 12 heads, d = 128: 489 us (1101 TFLOP/s; 565 us where the
// power limit lowers the clocks of a long run), against 331 for the products alone.  A test
// in the common block costs 2% of that, which is why values past the sequence are cleared
// inside the branch for blocks that the mask cuts.
// Rejected: one maximum a block guessed from the last one's (fewer instructions on the
// common path, but 27% more time for the test and the repeat behind it).
#include "window_tc.cuh"

namespace monarch {
namespace win {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 512;
constexpr int kSoftmaxRegs = 136, kEpilogueRegs = 128, kProducerRegs = 112;
static_assert(2 * kSoftmaxRegs + kEpilogueRegs + kProducerRegs == 4 * (65536 / kThreads),
              "the warpgroups' registers must add up to the launch's 128 per thread");

// Entries of the line: (pair, batch), all heads of one alike; CTAs that divide it.
constexpr int kMaxEntries = 512, kMaxCtas = 512;
// Segments of one CTA.
constexpr int kMaxSegments = 480;

// What one CTA does of one problem, as shared memory holds it: key blocks
// [first, first + nh) of the problem's.
struct Record {
    int unit;            // entry * H + head
    int first, nh;
    int sinks, window;   // blocks of the problem's sinks; first block of its window
    int len;             // keys of the problem's sequence, with the sign bit set where the
                         // problem's last block is among these
    int start;           // position of the sequence's first query
    __device__ __forceinline__ Sequence seq() const { return {len & 0x7fffffff, start}; }
    __device__ __forceinline__ bool ends() const { return len < 0; }
};
constexpr int kEnds = (int)0x80000000;

// Shared memory for a head of D columns (tiles of 128 rows).
template <int D> struct Layout {
    static constexpr uint32_t kTile = (D / 64) * kPanel;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = 2 * kTile;
    static constexpr uint32_t kV = kK + 2 * kTile;
    static constexpr uint32_t kL = kV + 2 * kTile;          // row sums [parity][tile][128]
    static constexpr uint32_t kStg = kL + 2048;             // epilogue: 4 warps x 32 rows x 128 B
    static_assert(kMaxEntries * sizeof(Sequence) <= 4 * 4096, "the sequences of the line");
    static constexpr uint32_t kLine = kStg + 4 * 4096;      // first chunk of each entry
    static constexpr uint32_t kList = kLine + (kMaxEntries + 1) * 4 + 12;
    static constexpr uint32_t kBar = kList + kMaxSegments * sizeof(Record);
    static constexpr uint32_t kSmem = kBar + 512 + 1024;    // + slack to align the base
    static_assert(kSmem <= (uint32_t)kMaxSmem, "window attention shared memory");
};

enum { kEvery, kReal, kLine };

struct FwdArgs {
    WinProblem p;
    int tiles;      // 128-row query tiles of a problem: 2, or 1 where pairs are fewer than SMs
    int npairs;     // problems a head
    int nprob;      // npairs * B * H
    int how;        // how the CTAs divide the problems
    // kLine: per slot (2 a CTA: a part that starts inside its problem, one that starts with
    // it) the problem and whether the part ends it, then maxima, row sums, sums
    int2 *meta;
    float *parts;
    __nv_bfloat16 *out;
    float *lse;     // or null
    int *status;
    long long limit;
    int stall;
};

// Floats of one slot: 256 maxima, 256 row sums, 256 rows of d sums.
__host__ __device__ constexpr int part_floats(int d) { return 512 + 256 * d; }

// Entry e of the line: pair npairs - 1 - e / B of batch e % B.  Later rows see more keys
// under a causal mask, so the longest problems come first and short ones fill the end.
__device__ __forceinline__ int entry_batch(const FwdArgs &a, int e) { return e % a.p.B; }
__device__ __forceinline__ int entry_row(const FwdArgs &a, int e) {
    return (a.npairs - 1 - e / a.p.B) * 128 * a.tiles;
}
// Its 64-key blocks.
__device__ __forceinline__ KeyTiles entry_tiles(const FwdArgs &a, int e, const Sequence &seq) {
    return key_tiles<64>(a.p, seq, entry_row(a, e), entry_row(a, e) + 128 * a.tiles);
}

// A segment, read from its record by each role.
struct Segment {
    int b, h, i0, first, nh, unit, turn, skip;
    bool begins, ends;
    __device__ __forceinline__ Segment(const FwdArgs &a, const Record &r) {
        const int e = r.unit / a.p.H;
        unit = r.unit;
        h = unit - e * a.p.H;
        b = entry_batch(a, e);
        i0 = entry_row(a, e);
        first = r.first;
        nh = r.nh;
        turn = r.sinks - first;   // blocks before it are the sinks', the others lie
        skip = r.window - r.sinks;   // `skip` further
        begins = first == 0;
        ends = r.ends();
    }
    __device__ __forceinline__ bool whole() const { return begins && ends; }
    __device__ __forceinline__ int slot() const { return 2 * blockIdx.x + (begins ? 1 : 0); }
    __device__ __forceinline__ int key(int i) const {
        return (first + i + (i < turn ? 0 : skip)) * 64;
    }
};

// The CTA's segments into `list`; returns their number.  Whole problems are dealt out
// forwards and backwards in turn, so that each CTA gets as many and long ones meet short
// ones: all of them (kEvery; nh = 0: no row sees a key), or those that have keys (kReal).
// The line (kLine): as many whole problems each as never exceed a CTA's share, CTA c the
// c-th of every gridDim (they start together, so the heads' keys are read from DRAM about
// once for all of them), then of the chunks behind those its share less what it has.
// lengths and starts are read once: what follows from them, the roles take from the list.
__device__ __forceinline__ int list_segments(const FwdArgs &a, int *line, Record *list,
                                             Sequence *seqs) {
    const WinProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ int count;
    auto problem = [&](int i) {
        return i * (int)gridDim.x + (int)(i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    };
    // (only the last round may be short of one)
    auto rounds_of = [&](int total) {
        const int rounds = (total + (int)gridDim.x - 1) / (int)gridDim.x;
        return rounds == 0 || problem(rounds - 1) < total ? rounds : rounds - 1;
    };
    auto whole_problem = [&](int unit, const Sequence &seq) {
        const KeyTiles kt = entry_tiles(a, unit / p.H, seq);
        return Record{unit, 0, kt.count(), kt.nA, kt.first, seq.len | kEnds, (int)seq.start};
    };
    if (a.how == kEvery) {
        const int n = rounds_of(a.nprob);
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int unit = problem(i);
            list[i] = whole_problem(unit, sequence(p, entry_batch(a, unit / p.H)));
        }
        return n;
    }
    const int entries = a.npairs * p.B;
    for (int b = threadIdx.x; b < p.B; b += kThreads) seqs[b] = sequence(p, b);
    __syncthreads();
    auto tiles_of = [&](int e) { return entry_tiles(a, e, seqs[entry_batch(a, e)]); };
    for (int e = threadIdx.x; e < entries; e += kThreads) {
        const int chunks = (tiles_of(e).count() + 1) / 2;
        line[e + 1] = (a.how == kLine ? chunks : min(chunks, 1)) * p.H;
    }
    if (threadIdx.x == 0) line[0] = 0;
    if (a.how == kLine && threadIdx.x < 2)
        a.meta[2 * blockIdx.x + threadIdx.x] = make_int2(-1, 0);
    __syncthreads();
    if (warp == 0) {
        int sum = 0, longest = 0;
        for (int e0 = 1; e0 <= entries; e0 += 32) {
            int x = e0 + lane <= entries ? line[e0 + lane] : 0;
            longest = max(longest, __reduce_max_sync(0xffffffffu, x) / p.H);
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, m);
                if (lane >= m) x += y;
            }
            if (e0 + lane <= entries) line[e0 + lane] = sum + x;
            sum += __shfl_sync(0xffffffffu, x, 31);
        }
        __syncwarp();   // lane 0 reads what the other lanes have written
        if (lane == 0 && a.how == kLine) {
            const int c = blockIdx.x, ctas = gridDim.x, whole = longest ? sum / ctas / longest : 0;
            // where problem i (entry i / H, head i % H) begins in the line
            auto begin = [&](int i) {
                const int e = i / p.H;
                return e == entries ? sum : line[e] + (line[e + 1] - line[e]) / p.H * (i - e * p.H);
            };
            const int rest = begin(whole * ctas);
            int at = rest + (int)((int64_t)sum * c / ctas), n = 0, e = 0;
            int end = rest + (int)((int64_t)sum * (c + 1) / ctas);
            for (int j = 0; j < whole; j++) {
                const int i = j * ctas + c;
                at -= begin(i) - begin(j * ctas);
                end -= begin(i + 1) - begin(j * ctas);
                const Record r = whole_problem(i, seqs[entry_batch(a, i / p.H)]);
                if (r.nh > 0) list[n++] = r;
            }
            while (at < end && n < kMaxSegments) {
                while (line[e + 1] <= at) e++;
                const KeyTiles kt = tiles_of(e);
                const Sequence &seq = seqs[entry_batch(a, e)];
                const int blocks = kt.count(), chunks = (blocks + 1) / 2;
                const int h = (at - line[e]) / chunks, c0 = at - line[e] - h * chunks;
                const int c1 = min(chunks, c0 + end - at);
                list[n++] = Record{e * p.H + h, 2 * c0, min(blocks, 2 * c1) - 2 * c0, kt.nA, kt.first,
                                   seq.len | (c1 == chunks ? kEnds : 0), (int)seq.start};
                at += c1 - c0;
            }
            count = n;
        }
    }
    __syncthreads();
    if (a.how == kLine) return count;
    const int n = rounds_of(line[entries]);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int x = problem(i);
        int lo = 0, hi = entries;   // the entry with line[e] <= x < line[e + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            (line[mid] <= x ? lo : hi) = mid;
        }
        list[i] = whole_problem(lo * p.H + (x - line[lo]), seqs[entry_batch(a, lo)]);
    }
    return n;
}

// Blocks j and j + 1 of a segment's keys or values to a stage: one box of 128 rows, or two
// of 64 where they are not neighbours (the sinks' last block) or the last is alone.
template <int D>
__device__ __forceinline__ void load_chunk(uint8_t *dst, const CUtensorMap *map64,
                                           const CUtensorMap *map128, const Segment &sg, int j,
                                           int G, uint64_t *bar) {
    const int blocks = min(2, sg.nh - j), row = sg.key(j);
    mbar_expect_tx(bar, blocks * Layout<D>::kTile / 2);
    if (blocks == 2 && sg.key(j + 1) == row + 64) {
        for (int pn = 0; pn < D / 64; pn++)
            tma_load_4d(dst + pn * kPanel, map128, pn * 64, row, sg.h / G, sg.b, bar);
        return;
    }
    for (int x = 0; x < blocks; x++)
        for (int pn = 0; pn < D / 64; pn++)
            tma_load_4d(dst + pn * kPanel + x * 64 * 128, map64, pn * 64, sg.key(j + x), sg.h / G,
                        sg.b, bar);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tc_window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmK128,
                     const __grid_constant__ CUtensorMap tmV128, FwdArgs a) {
    using L = Layout<D>;
    constexpr int PN = D / 64;
    constexpr uint32_t kTile = L::kTile;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = align1024(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kBar);
    uint64_t *q_full = bars + 0;     // [2 tiles]
    uint64_t *q_empty = bars + 2;    // [2 tiles]: the tile's last S product of a problem done
    uint64_t *k_full = bars + 4;     // [2 stages]
    uint64_t *k_empty = bars + 6;    // [2 stages], one commit from each issuer
    uint64_t *v_full = bars + 8;     // [2 stages]
    uint64_t *v_empty = bars + 10;   // [2 stages], one commit from each issuer
    uint64_t *s_full = bars + 12;    // [2 tiles][2 S buffers]
    uint64_t *p_full = bars + 16;    // [2 tiles][2 S buffers], one arrival per softmax warp
    uint64_t *o_full = bars + 20;    // [2 tiles]: the last PV product of a problem done
    uint64_t *o_free = bars + 22;    // [2 tiles], one arrival per epilogue warp
    uint64_t *l_full = bars + 24;    // [2 tiles], one arrival per softmax warp
    uint64_t *mma_done = bars + 26;
    uint64_t *stall_bar = bars + 27;   // never completed (fault injection)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 28);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 29);
    uint64_t *pv_done = bars + 30;   // [2 tiles]: one phase per PV product
    float *lsum = reinterpret_cast<float *>(sm + L::kL);   // [2][2][128]

    const WinProblem &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *line = reinterpret_cast<int *>(sm + L::kLine);

    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; t++) {
            mbar_init(q_full + t, 1);
            mbar_init(q_empty + t, 1);
            mbar_init(k_full + t, 1);
            mbar_init(k_empty + t, a.tiles);
            mbar_init(v_full + t, 1);
            mbar_init(v_empty + t, a.tiles);
            for (int b = 0; b < 2; b++) {
                mbar_init(s_full + 2 * t + b, 1);
                mbar_init(p_full + 2 * t + b, 4);
            }
            mbar_init(pv_done + t, 1);
            mbar_init(o_full + t, 1);
            mbar_init(o_free + t, 4);
            mbar_init(l_full + t, 4);
        }
        mbar_init(mma_done, a.tiles);
        mbar_init(stall_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 13) tmem_alloc(tmem_slot, 512);
    Record *list = reinterpret_cast<Record *>(sm + L::kList);
    // (the sequences lie where the epilogue stages its rows later)
    const int nseg = list_segments(a, line, list, reinterpret_cast<Sequence *>(sm + L::kStg));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx w{a.limit, a.status, abort_flag};
    // Every role takes the same segments; pc counts those with keys, as the barriers do.

    if (warp >= 12) {
        regs_dec<kProducerRegs>();
        if (warp == 12) {
            // ---------------- keys: a chunk as soon as the S products of two chunks
            // back are done
            int issued[2] = {0, 0}, jc = 0;
            bool ok = true;
            for (int si = 0; ok && si < nseg; si++) {
                const Segment sg(a, list[si]);
                if (sg.nh == 0) continue;
                for (int j = 0; j < sg.nh; j += 2, jc++) {
                    const int sk = jc & 1;
                    if (jc >= 2 && !wait_warp(k_empty + sk, ((jc >> 1) - 1) & 1, w)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0)
                        load_chunk<D>(sm + L::kK + sk * kTile, &tmK, &tmK128, sg, j, p.G, k_full + sk);
                    issued[sk]++;
                }
            }
            if (lane == 0)   // every issued copy lands before the CTA may exit
                for (int s = 0; s < 2; s++)
                    if (issued[s] > 0)
                        wait_phase_cleanup(k_full + s, (issued[s] - 1) & 1, kCleanupPolls);
        } else if (warp == 14) {
            // ---------------- queries, then values.  Every wait points at a product
            // that the issuers reach without these loads: a tile's last S of the
            // previous problem follows that problem's values in the issue order.
            int pc = 0, issued[2] = {0, 0}, jc = 0, qloads[2] = {0, 0};
            bool ok = true;
            for (int si = 0; ok && si < nseg; si++) {
                const Segment sg(a, list[si]);
                if (sg.nh == 0) continue;
                for (int t = 0; t < a.tiles; t++) {
                    if (pc > 0 && !wait_warp(q_empty + t, (pc - 1) & 1, w)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        mbar_expect_tx(q_full + t, kTile);
                        for (int pn = 0; pn < PN; pn++)
                            tma_load_4d(sm + L::kQ + t * kTile + pn * kPanel, &tmQ, pn * 64,
                                        sg.i0 + t * 128, sg.h, sg.b, q_full + t);
                    }
                    qloads[t]++;
                }
                if (!ok) break;
                pc++;
                for (int j = 0; j < sg.nh; j += 2, jc++) {
                    const int st = jc & 1;
                    if (jc >= 2 && !wait_warp(v_empty + st, ((jc >> 1) - 1) & 1, w)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0)
                        load_chunk<D>(sm + L::kV + st * kTile, &tmV, &tmV128, sg, j, p.G, v_full + st);
                    issued[st]++;
                }
            }
            if (lane == 0) {
                for (int t = 0; t < 2; t++)
                    if (qloads[t] > 0)
                        wait_phase_cleanup(q_full + t, (qloads[t] - 1) & 1, kCleanupPolls);
                for (int st = 0; st < 2; st++)
                    if (issued[st] > 0)
                        wait_phase_cleanup(v_full + st, (issued[st] - 1) & 1, kCleanupPolls);
            }
        } else {
            // ---------------- product issuers.  Half hc (over the CTA's problems) of
            // tile t uses S buffer hc & 1.  Order: S of the first two halves, then per
            // half PV(hc), S(hc + 2).  S(hc + 2) overwrites the columns that PV(hc)
            // reads as P: one thread's products execute in issue order.
            if (warp - 13 < 2 * a.tiles - 1 && elect_one()) {
            const int t = warp == 13 ? 0 : 1;
            constexpr uint32_t idS = idesc_bf16(128, 64, 0, 0);
            constexpr uint32_t idO = idesc_bf16(128, D, 0, 1);
            const uint64_t dQ = smem_desc_sw128(smem_u32(sm + L::kQ + t * kTile), 16, 1024);
            const uint64_t dK = smem_desc_sw128(smem_u32(sm + L::kK), 16, 1024);
            const uint64_t dV = smem_desc_sw128(smem_u32(sm + L::kV), kPanel, 1024);
            constexpr uint32_t kTileDesc = kTile >> 4, kHalfDesc = 64 * 128 >> 4;
            const uint32_t tS = tmem + t * 128, tO = tmem + 256 + t * 128;
            bool ok = !a.stall || wait_phase(stall_bar, 0, w);
            struct Cursor {
                int si, nh, pc, i, hc, jc0;   // segment, its blocks; block i, hc of all
            };
            auto find = [&](Cursor &c) {
                while (c.si < nseg && (c.nh = list[c.si].nh) == 0) c.si++;
            };
            auto advance = [&](Cursor &c) {
                c.hc++;
                if (++c.i == c.nh) {
                    c.i = 0;
                    c.jc0 += (c.nh + 1) / 2;
                    c.pc++;
                    c.si++;
                    find(c);
                }
            };
            auto issue_s = [&](const Cursor &c) -> bool {
                const int jc = c.jc0 + (c.i >> 1), sk = jc & 1, kh = c.i & 1, b = c.hc & 1;
                if (c.i == 0 && !wait_phase(q_full + t, c.pc & 1, w)) return false;
                if (kh == 0 && !wait_phase(k_full + sk, (jc >> 1) & 1, w)) return false;
                tc_fence_after();
                mma_head<D, 128>(tS + b * 64, dQ, dK + sk * kTileDesc + kh * kHalfDesc, idS);
                mma_commit(s_full + 2 * t + b);
                const bool last = c.i == c.nh - 1;
                if (kh == 1 || last) mma_commit(k_empty + sk);
                if (last) mma_commit(q_empty + t);
                return true;
            };
            auto issue_pv = [&](const Cursor &c) -> bool {
                const int jc = c.jc0 + (c.i >> 1), st = jc & 1, kh = c.i & 1, b = c.hc & 1;
                if (kh == 0 && !wait_phase(v_full + st, (jc >> 1) & 1, w)) return false;
                if (!wait_phase(p_full + 2 * t + b, (c.hc >> 1) & 1, w)) return false;
                // the first PV of a problem overwrites O: the epilogue must have read it
                if (c.i == 0 && c.pc > 0 && !wait_phase(o_free + t, (c.pc - 1) & 1, w)) return false;
                tc_fence_after();
                mma_block64<16>(tO, tS + b * 64, dV + st * kTileDesc + kh * kHalfDesc, idO,
                             c.i > 0 ? 1u : 0u);
                mma_commit(pv_done + t);
                const bool last = c.i == c.nh - 1;
                if (kh == 1 || last) mma_commit(v_empty + st);
                if (last) mma_commit(o_full + t);
                return true;
            };
            Cursor cs{0, 0, 0, 0, 0, 0};    // next S to issue
            find(cs);
            Cursor cp = cs;                 // next PV to issue
            for (int k = 0; ok && k < 2 && cs.si < nseg; k++) {
                ok = issue_s(cs);
                advance(cs);
            }
            while (ok && cp.si < nseg) {
                const bool more = cs.si < nseg;
                ok = issue_pv(cp) && (!more || issue_s(cs));
                if (more) advance(cs);
                advance(cp);
            }
            mma_commit(mma_done);
            wait_phase_cleanup(mma_done, 0, kCleanupPolls);
            }
            __syncwarp();
        }
    } else if (warp >= 8) {
        // ---------------- epilogue: O / l to bfloat16 rows
        regs_dec<kEpilogueRegs>();
        const int wq = warp & 3;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        bool ok = true;
        int pc = 0;
        for (int si = 0; ok && si < nseg; si++) {
            const Segment sg(a, list[si]);
            if (sg.nh == 0) continue;
            // these waits last as long as the whole segment, so their limit grows with it
            // (each block's own waits have the plain one and raise the abort flag)
            const WaitCtx whole{a.limit * (1 + sg.nh / 16), a.status, abort_flag};
            for (int t = 0; t < a.tiles; t++) {
                if (!wait_warp(o_full + t, pc & 1, whole) ||
                    !wait_warp(l_full + t, pc & 1, whole)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (!sg.whole()) {   // the unscaled sums, for the join
                    float *dst = a.parts + (int64_t)sg.slot() * part_floats(D) + 512 +
                                 (t * 128 + wq * 32 + lane) * D;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        tmem_ld32f(tmem + lane_off + 256 + t * 128 + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4 *>(dst + c + k) =
                                make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                    }
                    tc_fence_before();
                    mbar_arrive_warp(o_free + t);
                    continue;
                }
                const float total = lsum[((pc & 1) * 2 + t) * 128 + wq * 32 + lane];
                const float inv_l = 1.f / total;
                uint32_t pk[D / 2];
#pragma unroll
                for (int c = 0; c < D / 32; c++) {
                    float o[32];
                    tmem_ld32f(tmem + lane_off + 256 + t * 128 + c * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; k++)
                        pk[c * 16 + k] = total == 0.f ? 0u   // a row that sees nothing
                                                      : pack_bf16(o[2 * k] * inv_l,
                                                                  o[2 * k + 1] * inv_l);
                }
                tc_fence_before();
                mbar_arrive_warp(o_free + t);
                // the warp's 32 rows leave through shared memory, 128 bytes of a row at a
                // time, so each store instruction covers four runs of 128 bytes
                uint8_t *stg = sm + L::kStg + wq * 4096;
                const int m0 = sg.i0 + t * 128 + wq * 32;
                __nv_bfloat16 *const base = a.out + sg.b * p.o.batch + sg.h * p.o.head;
#pragma unroll
                for (int hf = 0; hf < PN; hf++) {
#pragma unroll
                    for (int c = 0; c < 8; c++)
                        *reinterpret_cast<uint4 *>(stg + lane * 128 + ((c + lane) & 7) * 16) =
                            make_uint4(pk[hf * 32 + 4 * c], pk[hf * 32 + 4 * c + 1],
                                       pk[hf * 32 + 4 * c + 2], pk[hf * 32 + 4 * c + 3]);
                    __syncwarp();
#pragma unroll
                    for (int rr = 0; rr < 8; rr++) {
                        const int row = rr * 4 + (lane >> 3), c = lane & 7;
                        const uint4 val =
                            *reinterpret_cast<const uint4 *>(stg + row * 128 + ((c + row) & 7) * 16);
                        // (d = 32 runs with D = 64: the columns past d are padding)
                        if (m0 + row < p.Nq && hf * 64 + c * 8 < p.d)
                            *reinterpret_cast<uint4 *>(base + (int64_t)(m0 + row) * p.o.token +
                                                       hf * 64 + c * 8) = val;
                    }
                    __syncwarp();
                }
            }
            pc++;
        }
    } else if (regs_inc<kSoftmaxRegs>(); (warp >> 2) < a.tiles) {
        // ---------------- softmax of tile t: one query row a thread
        const int t = warp >> 2, wq = warp & 3;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const uint32_t tS0 = tmem + lane_off + t * 128;
        const uint32_t tO = tmem + lane_off + 256 + t * 128;
        const float c1 = p.scale_log2;
        const uint64_t c2 = f2_pack(c1, c1);
        bool ok = true;
        int pc = 0, hc = 0, jc0 = 0;
        // rows of a pair that sees no key: zeros
        auto write_zeros = [&](int unit) {
            const int e = unit / p.H, h = unit % p.H, bb = entry_batch(a, e);
            const int m = entry_row(a, e) + t * 128 + wq * 32 + lane;
            if (m >= p.Nq) return;
            uint4 *row = reinterpret_cast<uint4 *>(a.out + bb * p.o.batch + h * p.o.head +
                                                   (int64_t)m * p.o.token);
            for (int c = 0; c < p.d / 8; c++) row[c] = make_uint4(0, 0, 0, 0);
            if (a.lse) a.lse[((int64_t)bb * p.H + h) * p.Nq + m] = -INFINITY;
        };
        for (int e = 0; a.how != kEvery && e < a.npairs * p.B; e++)   // (in no segment)
            if (line[e + 1] == line[e])
                for (int h = (blockIdx.x + e) % gridDim.x; h < p.H; h += gridDim.x)
                    write_zeros(e * p.H + h);
        for (int si = 0; ok && si < nseg; si++) {
            const Segment sg(a, list[si]);
            if (sg.nh == 0) {
                write_zeros(sg.unit);
                continue;
            }
            const int m = sg.i0 + t * 128 + wq * 32 + lane;
            const Sequence seq = list[si].seq();
            // a row that is not real takes every key of the sequence, so that its warp needs
            // no masks (its sums touch nothing else), and its row sum goes out as 0
            RowKeys rk = row_keys(p, seq, m);
            const bool real = rk.hi > 0;
            if (!real) rk = RowKeys{0, seq.len, 0};
            float m_run = -INFINITY, l_run = 0.f;
            for (int i = 0; i < sg.nh; i++, hc++) {
                const int b = hc & 1;
                if (!wait_warp(s_full + 2 * t + b, (hc >> 1) & 1, w)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tS = tS0 + b * 64;
                const int j0 = sg.key(i);
                float x[64];
                tmem_ld32f(tS, &x[0]);
                tmem_ld32f(tS + 32, &x[32]);
                tmem_wait_ld();
                const bool all = j0 + 64 <= rk.hi && (j0 >= rk.lo || j0 + 64 <= rk.sink);
                if (!__all_sync(0xffffffffu, all)) {
                    // bit k: the row sees key j0 + k
                    auto below = [](int n) -> uint64_t {
                        return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
                    };
                    const uint64_t see = below(rk.hi - j0) &
                                         (~below(rk.lo - j0) | below(rk.sink - j0));
                    const uint32_t see0 = (uint32_t)see, see1 = (uint32_t)(see >> 32);
#pragma unroll
                    for (int k = 0; k < 32; k++) {
                        x[k] = (see0 >> k) & 1 ? x[k] : -INFINITY;
                        x[k + 32] = (see1 >> k) & 1 ? x[k + 32] : -INFINITY;
                    }
                    if (j0 + 64 > seq.len) {   // (no row takes such a block whole)
                        // values past the sequence may hold anything, and 0 * NaN is NaN: they
                        // become zeros before this half's PV (both tiles write the same zeros)
                        const int jc = jc0 + (i >> 1), st = jc & 1;
                        if (!wait_warp(v_full + st, (jc >> 1) & 1, w)) {
                            ok = false;
                            break;
                        }
                        zero_rows(sm + L::kV + st * kTile + (i & 1) * 64 * 128,
                                  max(0, seq.len - j0), 64, PN, kPanel, wq * 32 + lane, 128);
                        fence_proxy_async_smem();
                    }
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 32; k++) mx4[k & 3] = fmax3(mx4[k & 3], x[2 * k], x[2 * k + 1]);
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                float alpha = 1.f;
                bool rescale = false;
                if ((mx - m_run) * c1 > 8.f) {   // (false for a row without keys so far)
                    alpha = fast_exp2((m_run - mx) * c1);
                    m_run = mx;
                    rescale = true;
                }
                const float mm = m_run == -INFINITY ? 0.f : m_run * c1;
                const uint64_t nmc2 = f2_pack(-mm, -mm);
                uint64_t sum2[4] = {0, 0, 0, 0};
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 32; k++) {
                    const uint64_t d2 = f2_fma(f2_pack(x[2 * k], x[2 * k + 1]), c2, nmc2);
                    float lo, hi;
                    f2_unpack(d2, lo, hi);
                    const uint64_t e2 = f2_pack(fast_exp2(lo), fast_exp2(hi));
                    sum2[k & 3] = f2_add(sum2[k & 3], e2);
                    float p0, p1;
                    f2_unpack(e2, p0, p1);
                    pk[k] = pack_bf16(p0, p1);
                }
                tmem_st32(tS, pk);   // P over the first 32 columns of the buffer
                float s0, s1;
                f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), s0, s1);
                l_run = l_run * alpha + (s0 + s1);
                if (i > 0 && __any_sync(0xffffffffu, rescale)) {
                    // O holds the products up to the previous half once that PV is done
                    if (!wait_warp(pv_done + t, (hc - 1) & 1, w)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 32; c++) {
                        float o[32];
                        tmem_ld32f(tO + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; k++) o[k] *= alpha;
                        tmem_st32f(tO + c * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive_warp(p_full + 2 * t + b);
            }
            if (!ok) break;
            jc0 += (sg.nh + 1) / 2;
            if (!real) m_run = -INFINITY, l_run = 0.f;
            if (!sg.whole()) {
                float *dst = a.parts + (int64_t)sg.slot() * part_floats(D) + t * 128 + wq * 32 + lane;
                dst[0] = m_run * c1;
                dst[256] = l_run;
                if (threadIdx.x == 0) a.meta[sg.slot()] = make_int2(sg.unit, sg.ends);
            } else if (a.lse && m < p.Nq)
                a.lse[((int64_t)sg.b * p.H + sg.h) * p.Nq + m] =
                    l_run == 0.f ? -INFINITY : (m_run * c1 + log2f(l_run)) * kLn2;
            // the row sums for the epilogue, once it has taken those of the last problem
            if (pc > 0 && !wait_warp(o_free + t, (pc - 1) & 1, w)) break;
            lsum[((pc & 1) * 2 + t) * 128 + wq * 32 + lane] = l_run;
            mbar_arrive_warp(l_full + t);
            pc++;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The parts of problems that a boundary cut.  Block (c, y): the problem whose first part
// CTA c made; 16 rows of it.  Parts in order, so the result does not vary.
template <int D>
__global__ void __launch_bounds__(256) window_join_kernel(FwdArgs a, int ctas) {
    const WinProblem &p = a.p;
    __shared__ int slots[kMaxCtas], parts;
    const int2 head = a.meta[2 * blockIdx.x + 1];
    if (head.x < 0) return;
    if (threadIdx.x < 32) {
        // its first part, then those of the CTAs behind (some may have had no chunk)
        int n = 1;
        bool more = true;
        if (threadIdx.x == 0) slots[0] = 2 * blockIdx.x + 1;
        for (int c0 = blockIdx.x + 1; more && c0 < ctas; c0 += 32) {
            const int c = c0 + threadIdx.x;
            const int2 m = c < ctas ? a.meta[2 * c] : make_int2(-1, 0);
            uint32_t mine = __ballot_sync(0xffffffffu, m.x == head.x);
            const uint32_t last = __ballot_sync(0xffffffffu, m.x == head.x && m.y);
            if (last) more = false, mine &= last | (last - 1);   // up to the one that ends it
            if ((mine >> threadIdx.x) & 1)
                slots[n + __popc(mine & ((1u << threadIdx.x) - 1))] = 2 * c;
            n += __popc(mine);
        }
        if (threadIdx.x == 0) parts = n;
    }
    __syncthreads();
    const int n = parts;
    const int b = entry_batch(a, head.x / p.H), i0 = entry_row(a, head.x / p.H), h = head.x % p.H;
    for (int at = threadIdx.x; at < 16 * (D / 4); at += 256) {
        const int row = blockIdx.y * 16 + at / (D / 4), col = at % (D / 4) * 4;
        const int m = i0 + row;
        if (m >= p.Nq || col >= p.d) continue;
        float mx = -INFINITY;
        for (int i = 0; i < n; i++) {
            mx = fmaxf(mx, a.parts[(int64_t)slots[i] * part_floats(D) + row]);
        }
        const float safe = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < n; i++) {
            const float *src = a.parts + (int64_t)slots[i] * part_floats(D);
            const float f = exp2f(src[row] - safe);
            const float4 v = *reinterpret_cast<const float4 *>(src + 512 + row * D + col);
            sum = fmaf(f, src[256 + row], sum);
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z);
            o.w = fmaf(f, v.w, o.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (sum == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<uint2 *>(a.out + b * p.o.batch + h * p.o.head + (int64_t)m * p.o.token + col) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (a.lse && col == 0)
            a.lse[((int64_t)b * p.H + h) * p.Nq + m] =
                sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
    }
}

// Whether the CTAs divide the line of all chunks.  Whole problems on `sms` CTAs take as many
// rounds of the longest problem as there are problems a CTA; the line takes the mean, and
// about ten chunks' time (20 us) for the parts and the join.  4680 queries
// that see 18720 keys, 12 heads (228 pairs of 147 chunks on 148 SMs): 620 us whole, 541 by
// the line alone, whose CTAs read 1.42 GB from DRAM, 497 with whole problems first (0.53
// GB).  Chunks are estimated from the tensors' sizes and the window, as the lengths are on
// the device.
bool use_line(const WinProblem &p, int nprob, int sms) {
    const int64_t entries = (int64_t)((p.Nq + 255) / 256) * p.B;
    if (entries > kMaxEntries || sms > kMaxCtas) return false;
    const int64_t chunks = most_keys(p, 256) / 128 + 1;
    // at most one more: a run of n keys meets at most n / 64 + 2 blocks, the sinks' and the
    // window's n / 64 + 3 together
    const int64_t bound = entries * p.H * (chunks + 1);
    if (bound >= (1LL << 31)) return false;
    // segments of a CTA: at most its chunks, and at most the problems
    if (min((int64_t)nprob, bound / sms + 1) > kMaxSegments) return false;
    const int64_t rounds = (nprob + sms - 1) / sms;
    return rounds * chunks - nprob * chunks / sms >= 10;
}

template <int D>
cudaError_t launch(const WinProblem &p, const void *q, const void *k, const void *v, FwdArgs a,
                   int sms, cudaStream_t stream) {
    CUtensorMap mq, mk, mv, mk128, mv128;
    if (!map_tokens(&mq, q, p.q, p.B, p.H, p.Nq, p.d, 128) ||
        !map_tokens(&mk, k, p.k, p.B, p.Hkv, p.Nk, p.d, 64) ||
        !map_tokens(&mv, v, p.v, p.B, p.Hkv, p.Nk, p.d, 64) ||
        !map_tokens(&mk128, k, p.k, p.B, p.Hkv, p.Nk, p.d, 128) ||
        !map_tokens(&mv128, v, p.v, p.B, p.Hkv, p.Nk, p.d, 128))
        return cudaErrorInvalidValue;
    cudaError_t e = tcs::set_smem(tc_window_fwd_kernel<D>, Layout<D>::kSmem);
    if (e != cudaSuccess) return e;
    // (a CTA lists at most kMaxSegments problems: beyond, more CTAs than SMs)
    const int grid =
        a.how == kLine ? sms : max(min(a.nprob, sms), (a.nprob + kMaxSegments - 1) / kMaxSegments);
    tc_window_fwd_kernel<D><<<grid, kThreads, Layout<D>::kSmem, stream>>>(mq, mk, mv, mk128,
                                                                              mv128, a);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.how != kLine) return e;
    window_join_kernel<D><<<dim3(grid, 16), 256, 0, stream>>>(a, grid);
    return cudaGetLastError();
}

size_t meta_bytes(int sms) { return ((size_t)sms * 2 * sizeof(int2) + 255) & ~(size_t)255; }

}  // namespace

size_t tc_forward_bytes(const WinProblem &p) {
    const int sms = tcs::sm_count();
    if (!use_line(p, (p.Nq + 255) / 256 * p.B * p.H, sms)) return 0;
    return meta_bytes(sms) + (size_t)sms * 2 * part_floats(p.d == 128 ? 128 : 64) * sizeof(float);
}

cudaError_t tc_forward(const WinProblem &p, const void *q, const void *k, const void *v, void *out,
                       float *lse, void *workspace, int *status, long long limit,
                       cudaStream_t stream) {
    const int sms = tcs::sm_count();
    FwdArgs a;
    a.p = p;
    a.how = use_line(p, (p.Nq + 255) / 256 * p.B * p.H, sms) ? kLine : kEvery;
    // A tile alone on its SM takes little more than half of a pair's time a key block
    // (the two tiles share the exponentials' units), so where the pairs are fewer than
    // the SMs single tiles finish sooner: two padded causal batches of 1023 tokens with 8
    // heads 27 -> 22 us.
    a.tiles = a.how == kLine || (p.Nq + 255) / 256 * p.B * p.H >= sms ? 2 : 1;
    a.npairs = (p.Nq + 128 * a.tiles - 1) / (128 * a.tiles);
    a.nprob = a.npairs * p.B * p.H;
    // Several rounds of a ragged batch: problems without keys would leave some CTAs one
    // round more than others (2 x 4001 tokens, the second sequence of 2667: 78.7 -> 75.2
    // us).  With one round the list of the others only delays the start (two short batches
    // 68 -> 72 us, forward and backward).
    if (a.how == kEvery && p.lengths && a.nprob > sms && (int64_t)a.npairs * p.B <= kMaxEntries)
        a.how = kReal;
    a.meta = (int2 *)workspace;
    a.parts = (float *)((char *)workspace + meta_bytes(sms));
    a.out = (__nv_bfloat16 *)out;
    a.lse = lse;
    a.status = status;
    a.limit = limit;
    a.stall = device_inject_stall();
    return p.d == 128 ? launch<128>(p, q, k, v, a, sms, stream)
                      : launch<64>(p, q, k, v, a, sms, stream);
}

}  // namespace win
}  // namespace monarch
