// product_host.cuh -- host side of product.cuh: how a product is laid out
// (tile, splits, ring depth), its tensor maps and its launch.
#pragma once

#include <atomic>
#include <cstring>

#include "product.cuh"

namespace pws {
namespace fused {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

// One product as an entry point asks for it.
struct Product {
    int64_t M = 0, N = 0, K = 0;        // output rows and columns, length of one K segment
    int segments = 1, problems = 1;
    bool gated = false, amn = false, bmn = false;
    bool may_split = false;
    // 2: A is a 16-bit value and its rounding remainder, M rows each (M counts
    // both); the two halves' outputs are added
    int halves = 1;
    int chunk = 0;                      // K blocks per accumulator hand-over; 0: a unit's
    bool operator==(const Product& o) const {
        return M == o.M && N == o.N && K == o.K && segments == o.segments && problems == o.problems &&
               gated == o.gated && amn == o.amn && bmn == o.bmn && may_split == o.may_split && halves == o.halves &&
               chunk == o.chunk;
    }
};

// How a launch of one or two products runs: one tile shape and ring for both.
struct Layout {
    int cg = 1, nw = 1, bn = 256, tile_n = 256, a_rows = 128;
    int stages = 0, boxes = 1, a_bytes = 0, box_bytes = 0, slot_bytes = 0, tx_bytes = 0;
    int first = 0;              // which product is the launch's first job
    int extra_rounds = 0;
    struct Part {
        int tiles_m = 0, tiles_n = 0, splits = 1, kb_per_split = 0, nkb0 = 0, nkb = 0;
    } part[2];
};

// Time of u0 units of t0 each followed by u1 units of t1 each, dealt to
// `groups` groups as Schedule does.
inline double makespan(int64_t u0, double t0, int64_t u1, double t1, int64_t groups, int* extra_rounds) {
    const int64_t rounds0 = u0 / groups, rest = u0 % groups, late = groups - rest;
    *extra_rounds = 0;
    if (u1 == 0) return static_cast<double>(rounds0 + (rest ? 1 : 0)) * t0;
    const int extra = rest ? static_cast<int>(t0 / t1 + 0.5) : 0;
    *extra_rounds = extra;
    const double early0 = static_cast<double>(rounds0 + (rest ? 1 : 0)) * t0, late0 = static_cast<double>(rounds0) * t0;
    if (extra * late >= u1) {
        const double b = late0 + static_cast<double>(cdiv(u1, late)) * t1;
        return b > early0 ? b : early0;
    }
    const int64_t left = u1 - extra * late, rounds = left / groups, rem = left % groups;
    const double a = rest ? early0 + static_cast<double>(rounds + (rem > late ? 1 : 0)) * t1 : 0.0;
    const double b = late0 + static_cast<double>(extra + rounds + (rem ? 1 : 0)) * t1;
    return a > b ? a : b;
}

// Chooses the tile (CTA pair or single CTA, accumulator width) and the K
// splits with the least estimated time, in SM clocks:
//   per K block   the larger of the multiplies (a tile of bn columns takes
//                 2 bn clocks, the wide one 1024), the copy into shared memory (about 50 bytes a
//                 clock and SM from L2) and a ring slot's share of one
//                 round trip (3000 clocks over the ring's depth), a slot's
//                 handling by the issuing thread (400), and a chunk's share of its
//                 hand-over to the epilogue (1200: one token's head of 50001 x 2048
//                 takes 37 us with the 112 columns this gives it, 50 with 48);
//   per unit      the larger of its K blocks and the epilogue of the unit
//                 before (1000 + 10 bn), and 300 clocks between units;
//   per launch    a fill and a last epilogue (1500 + that);
//   a split       the join's launch (4000) and its traffic (3000 bytes a clock).
inline Layout best_layout(const Product* pr, int n, int num_sms) {
    Layout best;
    double best_time = 1e300;
    int64_t rows = 0;
    for (int i = 0; i < n; ++i) rows = pr[i].M > rows ? pr[i].M : rows;
    for (int kind = 0; kind < (rows > BM_CTA ? 3 : 1); ++kind) {
        const int cg = kind ? 2 : 1, nw = kind == 2 ? 2 : 1;
        if (nw == 2 && !pr[0].bmn) continue;
        for (int bn = MAX_BN; bn >= (nw == 2 ? MAX_BN : 16); bn -= 16) {
            if (cg == 2 && (bn % 32 != 0 || bn < 64)) continue;
            if (pr[0].bmn && (bn / cg) % 64 != 0) continue;
            Layout l;
            l.cg = cg;
            l.nw = nw;
            l.bn = bn;
            l.tile_n = pr[0].gated ? bn / 2 : bn;
            // a short box for the tokens of a launch that has no more of them
            l.a_rows = BM_CTA;
            if (n == 1 && !pr[0].amn && cg == 1 && rows < BM_CTA) l.a_rows = static_cast<int>(round_up(rows, 8));
            l.a_bytes = l.a_rows * 128;         // (an MN-major A is two boxes of 64 x 64: as many)
            const int b_bytes = nw * (bn / cg) * 128;
            l.tx_bytes = l.a_bytes + b_bytes;
            l.box_bytes = static_cast<int>(round_up(l.tx_bytes, 1024));
            // Narrow tiles take several K blocks to a slot: a wait, a fence and
            // a commit per block cost the issuing thread about 400 clocks, more
            // than their multiplies.
            l.boxes = 1;
            if (cg == 1 && !pr[0].bmn)
                while (l.boxes < kMaxBoxes && 2 * bn * l.boxes < 400) l.boxes *= 2;
            l.slot_bytes = l.boxes * l.box_bytes;
            // the multiply reads 128 A rows from a slot's start: past a short
            // box it reads what follows (rows of D that are not stored), which
            // must still be the ring
            const int slack = l.a_rows < BM_CTA ? BM_CTA * 128 : 0;
            l.stages = (RING_BYTES - slack) / l.slot_bytes;
            if (l.stages > MAX_STAGES) l.stages = MAX_STAGES;
            if (nw == 2) l.stages = WIDE_STAGES;
            const int64_t groups = num_sms / cg;
            const double trip = 3000.0 / (l.stages * l.boxes), issue = 400.0 / l.boxes, epilogue = 1000.0 + 10.0 * bn * nw;
            double per_kb[2] = {0.0, 0.0};
            // each product's candidate splits: 1, 2, 4, ... up to a full wave of the GPU
            int64_t tiles[2] = {0, 0}, most[2] = {1, 1};
            for (int i = 0; i < n; ++i) {
                Layout::Part& q = l.part[i];
                // (rows of a box past the matrix are filled, not copied)
                const double copy = ((pr[i].M < BM_CTA ? pr[i].M : BM_CTA) * 128 + b_bytes) / 50.0;
                per_kb[i] = 2.0 * bn * nw;
                if (copy > per_kb[i]) per_kb[i] = copy;
                if (trip > per_kb[i]) per_kb[i] = trip;
                if (issue > per_kb[i]) per_kb[i] = issue;
                if (pr[i].chunk && 1200.0 / pr[i].chunk > per_kb[i]) per_kb[i] = 1200.0 / pr[i].chunk;
                q.tiles_m = static_cast<int>(cdiv(pr[i].M, BM_CTA * cg));
                q.tiles_n = static_cast<int>(cdiv(pr[i].N, nw * l.tile_n));
                q.nkb0 = static_cast<int>(cdiv(pr[i].K, BK));
                q.nkb = q.nkb0 * pr[i].segments;
                tiles[i] = static_cast<int64_t>(q.tiles_m) * q.tiles_n * pr[i].problems;
                if (pr[i].may_split && tiles[i] < groups) {
                    most[i] = groups / tiles[i];
                    if (most[i] > q.nkb / 4) most[i] = q.nkb / 4 > 0 ? q.nkb / 4 : 1;
                }
            }
            const auto more = [](int64_t s, int64_t top) { return s >= top ? top + 1 : (2 * s < top ? 2 * s : top); };
            for (int64_t s0 = 1; s0 <= most[0]; s0 = more(s0, most[0])) {
                for (int64_t s1 = 1; s1 <= most[1]; s1 = more(s1, most[1])) {
                    int64_t units[2] = {0, 0};
                    double t[2] = {0.0, 1.0}, time = 1500.0 + epilogue;
                    bool joins = false, long_enough = true;
                    for (int i = 0; i < n; ++i) {
                        Layout::Part& q = l.part[i];
                        q.kb_per_split = static_cast<int>(cdiv(q.nkb, i ? s1 : s0));
                        q.splits = static_cast<int>(cdiv(q.nkb, q.kb_per_split));
                        if (q.kb_per_split < kWideBlocks) long_enough = false;
                        units[i] = tiles[i] * q.splits;
                        t[i] = q.kb_per_split * per_kb[i];
                        if (t[i] < epilogue) t[i] = epilogue;
                        t[i] += 300.0;
                        if (q.splits > 1 || pr[i].halves > 1) {
                            joins = true;
                            time += 8.0 * q.splits * pr[i].M * pr[i].N * pr[i].problems / 3000.0;
                        }
                    }
                    if (nw == 2 && !long_enough) continue;
                    if (joins) time += 4000.0;
                    l.first = n == 2 && t[1] > t[0] ? 1 : 0;
                    const int a = l.first, b = 1 - l.first;
                    time += makespan(units[a], t[a], units[b], t[b], groups, &l.extra_rounds);
                    if (time < best_time) {
                        best_time = time;
                        best = l;
                    }
                }
            }
        }
    }
    return best;
}

// best_layout, remembered for the last few sizes a host thread asked for: the
// search takes microseconds, as long as the launch itself.
inline Layout choose_layout(const Product* pr, int n, int num_sms) {
    struct Entry {
        Product pr[2];
        int n = 0, num_sms = 0;
        Layout l;
    };
    constexpr int kEntries = 16;
    static thread_local Entry cache[kEntries];
    static thread_local int next = 0;
    for (const Entry& e : cache)
        if (e.n == n && e.num_sms == num_sms && e.pr[0] == pr[0] && (n == 1 || e.pr[1] == pr[1])) return e.l;
    Entry& e = cache[next];
    next = (next + 1) % kEntries;
    e.n = n;
    e.num_sms = num_sms;
    for (int i = 0; i < n; ++i) e.pr[i] = pr[i];
    e.l = best_layout(pr, n, num_sms);
    return e.l;
}
inline Layout choose_layout(const Product& pr, int num_sms) { return choose_layout(&pr, 1, num_sms); }

// fp32 partial sums of a split product: rows padded to 16 bytes.
inline int64_t ld32_of(int64_t N) { return round_up(N, 4); }

// Whether the tensor memory accelerator can address rows of `ld` 16-bit elements at p.
inline bool tma_ok(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }

// Tensor map of an operand: K-major, `mn` rows of K elements, a box of
// box_rows rows; or MN-major, K rows of `mn` elements, a box of 64 x 64.
inline bool operand_map(CUtensorMap* map, const void* p, bool mn_major, int64_t mn, int64_t K, int64_t ld,
                        int box_rows) {
    return mn_major ? encode_tmap_f16_2d(map, p, mn, K, ld * 2, 64, BK)
                    : encode_tmap_f16_2d(map, p, K, mn, ld * 2, BK, box_rows);
}

// The parts of Params that every epilogue shares.
inline Params base_params(const Layout& l, int type, const DeviceInfo& info, cudaStream_t stream) {
    Params p;
    memset(&p, 0, sizeof(p));
    p.extra_rounds = l.extra_rounds;
    p.bn = l.bn;
    p.tile_n = l.tile_n;
    p.stages = l.stages;
    p.boxes = l.boxes;
    p.box_bytes = l.box_bytes;
    p.a_bytes = l.a_bytes;
    p.slot_bytes = l.slot_bytes;
    p.tx_bytes = l.tx_bytes;
    p.bf16 = type == GEMM_TYPE_BFLOAT;
    p.flags = debug_flags();
    p.timeout_ns = wait_timeout_ns();
    p.status = status_word(info, stream);
    return p;
}

// A product's operands: a[2 * problem + segment], and b[segment] (one b for
// both segments where A is MN-major); a null entry repeats the first.
struct Operands {
    const void* a[4] = {nullptr, nullptr, nullptr, nullptr};
    int64_t lda = 0;
    const void* b[2] = {nullptr, nullptr};
    int64_t ldb = 0;
};

// Fills job `at` of a launch (the first uses maps 0 on, the second those after
// the first's).
inline bool set_job(Params* p, Maps* maps, int at, const Product& pr, const Layout& l, const Layout::Part& part,
                    const Operands& op) {
    p->chunk = pr.chunk ? pr.chunk : 1 << 30;
    Job& j = p->job[at];
    j.M = static_cast<int>(pr.M);
    j.N = static_cast<int>(pr.N);
    j.nkb0 = part.nkb0;
    j.nkb = part.nkb;
    j.tiles_m = part.tiles_m;
    j.tiles_n = part.tiles_n;
    j.num_tiles = part.tiles_m * part.tiles_n * pr.problems;
    j.kb_per_split = part.kb_per_split;
    j.units = j.num_tiles * part.splits;
    j.amn = pr.amn;
    j.b_seg = pr.amn ? 0 : 1;
    // instruction descriptor: fp32 accumulator, operand types, operands'
    // majors, N >> 3, M >> 4
    const uint32_t t = p->bf16 ? 1u : 0u;
    j.idesc = (1u << 4) | (t << 7) | (t << 10) | ((pr.amn ? 1u : 0u) << 15) | ((pr.bmn ? 1u : 0u) << 16) |
              (static_cast<uint32_t>(l.bn >> 3) << 17) | (static_cast<uint32_t>((BM_CTA * l.cg) >> 4) << 24);
    // the second of two jobs: MN-major A takes four A maps, one B and two
    // outputs, K-major A two, two and one
    if (at == 1) {
        const Job& f = p->job[0];
        j.a_map = f.amn ? 4 : 2;
        j.b_map = f.amn ? 1 : 2;
        j.c_map = f.amn ? 2 : 1;
    }
    const int na = at == 0 && !pr.amn ? 2 : (pr.amn ? 4 : 2), nb = pr.amn ? 1 : 2;
    for (int i = 0; i < na; ++i) {
        CUtensorMap* m = &maps->a[j.a_map + i];
        if (i > 0 && !op.a[i]) *m = maps->a[j.a_map];
        else if (!operand_map(m, op.a[i], pr.amn, pr.M, pr.K, op.lda, l.a_rows)) return false;
    }
    const int b_box = pr.gated ? l.tile_n : l.bn / l.cg;
    for (int i = 0; i < nb; ++i) {
        CUtensorMap* m = &maps->b[j.b_map + i];
        if (i > 0 && !op.b[i]) *m = maps->b[j.b_map];
        else if (!operand_map(m, op.b[i], pr.bmn, pr.N, pr.K, op.ldb, b_box)) return false;
    }
    return true;
}

// A 16-bit output's store map; false where its epilogue has to store directly.
inline bool output_map(CUtensorMap* map, const Layout& l, const void* out, int64_t M, int64_t N, int64_t ld) {
    if (!tma_ok(out, ld) || l.tile_n < EPI_COLS) return false;
    return encode_tmap_f16_2d(map, out, N, M, ld * 2, EPI_COLS, 32);
}

template <int CG, int EPI, int NW>
int launch_cg(const Maps& maps, const Params& p, const DeviceInfo& info, cudaStream_t stream) {
    auto kern = product_kernel<CG, EPI, NW>;
    static std::atomic<int> capacity[64] = {};
    if (info.device < 0 || info.device >= 64) return GEMM_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1] = pdl_attribute();
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.attrs = attr;
    int cap = capacity[info.device].load(std::memory_order_relaxed);
    if (cap == 0) {
        // concurrent first calls compute and store the same value
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_LAUNCH;
        }
        cap = info.num_sms;
        if (CG == 2) {
            cfg.numAttrs = 1;
            cfg.gridDim = dim3(2 * info.num_sms, 1, 1);
            if (cudaOccupancyMaxActiveClusters(&cap, kern, &cfg) != cudaSuccess || cap <= 0) {
                cudaGetLastError();
                cap = info.num_sms / 2;
            }
        }
        capacity[info.device].store(cap, std::memory_order_relaxed);
    }
    const int units = p.job[0].units + p.job[1].units;
    const int groups = units < cap ? units : cap;
    cfg.gridDim = dim3(CG * groups, 1, 1);
    cfg.stream = stream;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, maps, p) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

template <int EPI>
int launch_product(const Layout& l, const Maps& maps, const Params& p, const DeviceInfo& info, cudaStream_t stream) {
    if constexpr (EPI == kEpiStore)
        if (l.nw == 2) return launch_cg<2, EPI, 2>(maps, p, info, stream);
    return l.cg == 2 ? launch_cg<2, EPI, 1>(maps, p, info, stream) : launch_cg<1, EPI, 1>(maps, p, info, stream);
}

// Hands out 256-byte aligned parts of a workspace; with no base it only counts.
struct Carver {
    char* base = nullptr;
    size_t used = 0;
    template <typename T>
    T* take(int64_t count) {
        const size_t at = used;
        used += (static_cast<size_t>(count) * sizeof(T) + 255) / 256 * 256;
        return base ? reinterpret_cast<T*>(base + at) : nullptr;
    }
};

// An operand TMA cannot address is copied once to rows of a multiple of 64
// elements (128-byte rows) in the workspace; `ld` becomes the copy's.
struct Source {
    const void* ptr = nullptr;
    int64_t ld = 0;
    uint16_t* copy = nullptr;
    bool repack = false;
};

inline Source source_of(const void* p, int64_t rows, int64_t cols, bool repack, Carver* c) {
    Source s;
    s.ptr = p;
    s.ld = cols;
    s.repack = repack;
    if (repack) {
        s.ld = round_up(cols, 64);
        s.copy = c->take<uint16_t>(rows * s.ld);
    }
    return s;
}

// Copies the rows of the sources that need it, in one launch (sources of
// `cols` columns each); their pointers are then TMA's to read.
struct Fill {
    Source* s;
    int64_t rows;
};
int fill_sources(const Fill (&f)[3], int64_t cols, cudaStream_t stream);

// ---- the backward products (gemm_bwd.cu)

// Few rows: up to here a 16-bit gradient that the tensor cores multiply comes
// with its rounding remainder as a second 16-bit value, since few rows average
// no rounding out: twice the rows (dx) or tokens (dW) of a product whose time
// is the weights' bytes.  Both halves' rows fit one CTA's 128.
constexpr int64_t kFewRows = 64;

// fp32 values a product's partial sums take.
inline int64_t split_floats(const Product& pr, const Layout::Part& part) {
    return part.splits > 1 || pr.halves > 1 ? part.splits * pr.problems * pr.M * ld32_of(pr.N) : 0;
}

// A backward product and where it goes: scale (acc_in + A B^T) to 16 bits at
// out16[problem] (rows N apart), or acc_in + A B^T in fp32 at acc_out (rows
// ld32_of(N) apart).
struct StoreProduct {
    Product pr;
    Operands op;
    void* out16[2] = {nullptr, nullptr};
    float* acc_out = nullptr;
    const float* acc_in = nullptr;
    const float* scale = nullptr;
    float* partial = nullptr;       // split_floats() floats
};
// One launch for the n (1 or 2) products, and one that joins their splits.
// Of two products, one has K-major A and the other MN-major A.
int run_store_products(const StoreProduct* sp, int n, const Layout& l, int type, const DeviceInfo& info,
                       cudaStream_t stream);

// ---- argument checks

// Rows and columns are counted in an int, and a tile's end may lie up to 512
// past the last of them.
constexpr int64_t kMaxSize = (1ll << 31) - 1024;
inline bool bad_size(int64_t n) { return n < 0 || n > kMaxSize; }
inline bool odd_address(const void* p) { return reinterpret_cast<uintptr_t>(p) & 1u; }
// accumulator tiles are counted in an int
inline bool too_many_tiles(int64_t rows, int64_t cols) { return cdiv(rows, 128) * cdiv(cols, 16) >= (1ll << 31); }

struct Range {
    const void* p;
    uint64_t bytes;
};
// Whether any output overlaps an input or another output.
template <int NI, int NO>
bool overlaps(const Range (&in)[NI], const Range (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        if (!out[i].p) continue;
        for (int j = 0; j < NI; ++j)
            if (in[j].p && ranges_overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
        for (int j = 0; j < i; ++j)
            if (out[j].p && ranges_overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
    }
    return false;
}
// Whether a call's workspace will do: there where needed, aligned, large
// enough, and apart from what the call reads and writes.
template <int NI, int NO>
bool workspace_ok(const void* ws, int64_t bytes, size_t need, const Range (&in)[NI], const Range (&out)[NO]) {
    if (need == 0) return true;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || bytes < static_cast<int64_t>(need)) return false;
    const Range w[1] = {{ws, need}};
    return !overlaps(in, w) && !overlaps(out, w);
}
inline uint64_t bytes16(int64_t a, int64_t b) { return static_cast<uint64_t>(a) * static_cast<uint64_t>(b) * 2u; }

}  // namespace fused
}  // namespace pws
