// One-token attention by warps on their own: each takes items of one request, key/value
// head (and chunk of its query heads) and up to `split` tiles of its tokens, fetches their
// keys and values into a ring of its own and leaves a part (maximum, sum, unnormalised
// outputs) that launch_join (k_shared.cu) puts together with the other parts of the head.
// The products are those of k_attend.cuh.
//
// What bounds it: memory, and for short rows the chain from a request's length over its
// pages to its first keys.  In k_attend.cuh a CTA's warps share every row, which ends with
// two of their barriers and a join in shared memory, about 3 us of its time; here a row's
// end is a warp's own and the others go on, and a warp's next items are on their way while
// it computes this one.  Behind shared beginnings of k_shared.cu's cases (device time of
// the three launches in us, by CTAs and by warps): 64 requests 44.5 and 40.8, 250 of an
// e4m3 cache 73.8 and 64.1, 32 on a long document 113 and 109.  Long rows are the CTAs':
// 200 requests of 8000 tokens 195 us against 231.
#include "k_attend.cuh"

namespace scute {

namespace {

// Eight warps on an SM, whose rings are three tiles: twelve with two tiles 42.3 us (64
// requests) and 61.9 (250, e4m3).
constexpr int OWN_WARPS = 4;           // of a CTA
constexpr int OWN_CTAS = 2;            // of an SM, at most
constexpr int OWN_RING = 6;            // tiles of a warp's ring, at most
// Of an item that is not a row's last: with 2 the 64 requests take 42.3 us and the 250
// 64.6, with 8 43.7 and 73.0.
constexpr int LEAST_TILES = 4;

// Tokens that a request sees, in tiles of positions first .. len - 1 (k_attend.cuh).
template <int MODE>
__device__ __forceinline__ int tiles_of(const AttendArgs &a, int r, int tt, Seen *y, bool *bad) {
    *y = seen_of<MODE>(a, r, tt, bad);
    return y->len > y->first ? (y->len - y->first + tt - 1) / tt : 0;
}

// Walks the tiles of a warp's items: every `step`-th item of the batch.
template <int MODE, int TT>
struct Cursor {
    const AttendArgs &a;
    const int *items_at;             // items of one head's rows of the requests before
    int hz, Z, split, step, item, items;
    int r, hk, z, part;              // the item: its row, and which of the row's parts it is
    Seen seen;
    int pos, stop;                   // positions of the tile, and the item's end

    __device__ __forceinline__ Cursor(const AttendArgs &args, const int *at, int z_chunks, int tiles, int warp, int warps)
        : a(args), items_at(at), Z(z_chunks), split(tiles), step(warps), item(warp) {
        hz = a.kv.heads * Z;
        items = at[a.n_req] * hz;
        open();
    }
    __device__ __forceinline__ bool more() const { return item < items; }
    __device__ __forceinline__ void open() {
        if (!more()) return;
        int lo = 0, hi = a.n_req - 1;                  // the last request whose items begin at this one or before
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((long long)items_at[mid] * hz <= item) lo = mid;
            else hi = mid - 1;
        }
        r = lo;
        const int parts = items_at[r + 1] - items_at[r], in = item - items_at[r] * hz, row = in / parts;
        part = in - row * parts;
        hk = row / Z;
        z = row - hk * Z;
        bool bad;
        tiles_of<MODE>(a, r, TT, &seen, &bad);
        pos = seen.first + part * split * TT;
        stop = min(seen.len, pos + split * TT);
    }
    // On to the next tile; whether it is another item's.
    __device__ __forceinline__ bool next() {
        pos += TT;
        if (pos < stop) return false;
        item += step;
        open();
        return true;
    }
};

template <typename M, int DC>
struct OwnShape {
    static constexpr int TILE = 2 * M::TT * M::ROW;
    static constexpr int WARP = 2 * M::HC * 4 + OWN_RING * 4;       // of a warp, beside its ring
    static constexpr int WARP_BYTES = (WARP + 127) / 128 * 128;
    static size_t smem(int ring, int n_req) { return (size_t)OWN_WARPS * (ring * TILE + WARP_BYTES) + 4 * ((size_t)n_req + 1) + 256; }
};

template <typename M, int DC, int MODE>
__global__ void __launch_bounds__(32 * OWN_WARPS, OWN_CTAS) attend_own_kernel(const AttendArgs a, int ring) {
    using S = OwnShape<M, DC>;
    constexpr int TT = M::TT, HC = M::HC, ESZ = M::ESZ, ROW = M::ROW;
    constexpr unsigned ALL = 0xffffffffu;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int warp_sum[OWN_WARPS + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.kv.dim, row_bytes = D * ESZ;
    uint8_t *const mine = smem + (size_t)warp * (ring * S::TILE + S::WARP_BYTES), *const extra = mine + ring * S::TILE;
    float *const s_m = reinterpret_cast<float *>(extra), *const s_l = s_m + HC;
    volatile unsigned *const s_ok = reinterpret_cast<unsigned *>(s_l + HC);
    int *const items_at = reinterpret_cast<int *>(smem + (size_t)OWN_WARPS * (ring * S::TILE + S::WARP_BYTES));
    const uint32_t ring_at = ptx::smem_u32(mine);
    // behind a head's elements every row of a tile stays zero
    if (row_bytes < ROW)
        for (int i = lane; i < ring * S::TILE / 16; i += 32) reinterpret_cast<uint4 *>(mine)[i] = make_uint4(0, 0, 0, 0);
    // (with shared beginnings the launch before is k_shared.cu's, which has waited for what
    // this one reads: only this one's end waits for it, for launch_join's sake)
    if constexpr (MODE != SHARED) ptx::grid_dep_wait();
    ptx::grid_dep_launch();

    // ------------------------------------------------ the plan: tiles of an item, items of every request
    const int n = a.n_req, Z = (a.group + HC - 1) / HC, hz = a.kv.heads * Z, warps = gridDim.x * OWN_WARPS;
    const int per = (n + 32 * OWN_WARPS - 1) / (32 * OWN_WARPS), r0 = min(n, (int)threadIdx.x * per), r1 = min(n, r0 + per);
    auto exclusive = [&](int x, int *total) {
        int inc = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(ALL, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < OWN_WARPS; ++w) {
            if (w < warp) before += warp_sum[w];
            all += warp_sum[w];
        }
        __syncthreads();
        *total = all;
        return before + inc - x;
    };
    bool any = false;
    int sum = 0, tiles;
#pragma unroll 4
    for (int r = threadIdx.x; r < n; r += 32 * OWN_WARPS) {
        bool bad;
        Seen seen;
        items_at[r] = tiles_of<MODE>(a, r, TT, &seen, &bad);
        any |= bad;
    }
    __syncthreads();
    for (int r = r0; r < r1; ++r) sum += items_at[r];
    if (any && blockIdx.x == 0) atomicOr(a.status, STATUS_PAGES);
    exclusive(sum, &tiles);
    // as many tiles as make two items of every warp (so that parts of rows are at most that
    // many more than rows)
    const int split = (int)max((long long)LEAST_TILES, quotient((long long)tiles * hz + 2 * warps - 1, 2 * warps));
    sum = 0;
    for (int r = r0; r < r1; ++r) sum += (items_at[r] + split - 1) / split;
    int at = exclusive(sum, &tiles);
    for (int r = r0; r < r1; ++r) {
        const int t = (items_at[r] + split - 1) / split;
        items_at[r] = at;
        at += t;
    }
    if (r1 == n && r0 < n) items_at[n] = at;
    __syncthreads();
    if (blockIdx.x == 0)
        for (int r = threadIdx.x; r <= n; r += 32 * OWN_WARPS) a.own_at[r] = items_at[r];

    // ------------------------------------------------ the warp's items
    constexpr int LR = ROW >= 512 ? 32 : ROW / 16, RI = 32 / LR, SUB = TT < 16 ? TT : 16;
    static_assert(ROW < 512, "a row is an instruction's part");
    const int piece = lane % LR, row0 = lane / LR;
    const bool here = piece * 16 < row_bytes;
    const long long tok_bytes = a.kv.token_stride * ESZ;
    const uint32_t lane_at = place_of<ROW>(row0, piece);
    const uint64_t policy = ptx::make_policy_evict_first();
    const int gw = blockIdx.x * OWN_WARPS + warp;
    Cursor<MODE, TT> f(a, items_at, Z, split, gw, warps);       // the tile to be fetched
    bool wrong = false;
    int f_slot = 0;
    auto page_of = [&] {                                        // of this lane's token of that tile
        const int i = f.pos + lane, token = token_of<MODE>(f.seen, i);
        return lane < TT && i < f.stop && token >= 0
                   ? a.kv.table[f.r * a.kv.table_stride + (a.page_shift >= 0 ? token >> a.page_shift : token / a.kv.page_size)] : -1;
    };
    int page = f.more() ? page_of() : -1;
    auto fetch = [&] {
        if (f.more()) {
            const int i = f.pos + lane, token = token_of<MODE>(f.seen, i);
            long long place = -1;
            if (lane < TT && i < f.stop && token >= 0) {
                if (page < 0 || page >= a.kv.n_pages) {
                    wrong = true;
                } else {
                    const int in = a.page_shift >= 0 ? token & (a.kv.page_size - 1) : token % a.kv.page_size;
                    place = ((long long)page * a.kv.page_stride + (long long)in * a.kv.token_stride) * ESZ;
                }
            }
            const unsigned ok = __ballot_sync(ALL, place >= 0);
            if (lane == 0) s_ok[f_slot] = ok;
            const char *kb = reinterpret_cast<const char *>(a.kv.k) + f.hk * a.kv.head_stride * ESZ;
            const char *vb = reinterpret_cast<const char *>(a.kv.v) + f.hk * a.kv.head_stride * ESZ;
            const uint32_t kd = ring_at + f_slot * S::TILE, vd = kd + TT * ROW;
#pragma unroll
            for (int u = 0; u < TT / SUB; ++u) {
                const int g = u * SUB;
                const long long place0 = __shfl_sync(ALL, place, g);
                // rows that lie in one page step by the token's stride
                if (__all_sync(ALL, lane / SUB != u || (place >= 0 && place == place0 + (lane - g) * tok_bytes))) {
                    const long long from = place0 + row0 * tok_bytes + piece * 16;
                    const char *ks = kb + from, *vs = vb + from;
                    if (here) {
#pragma unroll
                        for (int k = g / RI; k < (g + SUB) / RI; ++k) {
                            const uint32_t to = k * RI * ROW + (lane_at ^ turn_of<ROW>(k * RI));
                            copy16(kd + to, ks, policy);
                            copy16(vd + to, vs, policy);
                            ks += RI * tok_bytes;
                            vs += RI * tok_bytes;
                        }
                    }
                } else {
#pragma unroll 2
                    for (int k = g / RI; k < (g + SUB) / RI; ++k) {
                        const int row = k * RI + row0;
                        const long long p = __shfl_sync(ALL, place, row);
                        const uint32_t to = place_of<ROW>(row, piece);
                        if (here) {
                            copy16(kd + to, p >= 0 ? kb + p + piece * 16 : kb, p >= 0, policy);
                            copy16(vd + to, p >= 0 ? vb + p + piece * 16 : vb, p >= 0, policy);
                        }
                    }
                }
            }
            if (++f_slot == ring) f_slot = 0;
            f.next();
            if (f.more()) page = page_of();
        }
        ptx::cp_async_commit();                                 // (a group for every step, so that they can be counted)
    };
    M math(lane, 0);
    Cursor<MODE, TT> w(a, items_at, Z, split, gw, warps);       // the tile to be computed
    // the next item's queries, asked for when this one's are taken
    uint4 ahead[M::NQ][M::KP][M::QE];
    auto ask = [&](const Cursor<MODE, TT> &y) {
        const int h0 = y.hk * a.group + y.z * HC;
        if (y.more())
            math.read_queries(reinterpret_cast<const __nv_bfloat16 *>(a.q) + y.r * a.q_stride + (long long)h0 * D, min(HC, a.group - y.z * HC), D, ahead);
    };
    ask(w);
    for (int k = 0; k < ring - 1; ++k) fetch();
    int slot = 0;
    while (w.more()) {
        const int h0 = w.hk * a.group + w.z * HC, nh = min(HC, a.group - w.z * HC);
        const long long part_row = (long long)(items_at[w.r] + w.part) * a.q_heads + h0;
        const float scale = (a.kv.k_scale ? a.kv.k_scale[w.hk] : 1.f) * a.scale;
        math.queries(ahead, a.softcap > 0.f ? scale : scale * LOG2E);
        const int last = (w.stop - w.pos + TT - 1) / TT;
        w.item += w.step;
        w.open();
        ask(w);
        math.reset();
        for (int k = 0; k < last; ++k) {
            fetch();
            // all but the last ring - 1 steps' copies have arrived
            switch (ring) {
                case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
                case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
                case 4: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
                case 5: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
                default: asm volatile("cp.async.wait_group 5;" ::: "memory");
            }
            __syncwarp();
            const unsigned ok = s_ok[slot];
            const uint32_t kd = ring_at + slot * S::TILE;
            math.tile(kd, kd + TT * ROW, ok, a.softcap, [] { __syncwarp(); });
            if (++slot == ring) slot = 0;
        }
        math.stats(s_m, s_l);
        __syncwarp();
        if (lane < nh) a.stat[part_row + lane] = make_float2(s_m[lane], s_l[lane]);
        math.part(a.part_o + part_row * D, D, nh);
        __syncwarp();
    }
    if (__any_sync(ALL, wrong) && lane == 0) atomicOr(a.status, STATUS_PAGES);
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (MODE == SHARED) ptx::grid_dep_wait();
}

template <typename M, int DC, int MODE>
cudaError_t launch_own(const AttendArgs &a, int num_sms, cudaStream_t st) {
    using S = OwnShape<M, DC>;
    static std::atomic<unsigned long long> done{0};
    const auto kernel = attend_own_kernel<M, DC, MODE>;
    const cudaError_t e = allow_max_dynamic_smem(kernel, done);
    if (e != cudaSuccess) return e;
    // fewer CTAs on an SM where a large batch's list leaves too little room for their rings
    int per_sm = OWN_CTAS, ring = 0;
    for (; per_sm >= 1; --per_sm) {
        const long long room = (228 / per_sm - 1) * 1024 - (long long)S::smem(0, a.n_req) - 64;
        ring = (int)(room / (OWN_WARPS * S::TILE));
        if (ring >= 2) break;
    }
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    if (ring > OWN_RING) ring = OWN_RING;
    return launch_chained(kernel, num_sms * per_sm, 32 * OWN_WARPS, S::smem(ring, a.n_req), st, a, ring);
}
template <bool FP8, int MODE>
cudaError_t launch_own_type(const AttendArgs &a, int num_sms, cudaStream_t st) {
    const bool wide = a.group > 8;
    if (a.kv.dim > 64)
        return wide ? launch_own<MmaMath<FP8, 128, 2>, 128, MODE>(a, num_sms, st) : launch_own<MmaMath<FP8, 128, 1>, 128, MODE>(a, num_sms, st);
    return wide ? launch_own<MmaMath<FP8, 64, 2>, 64, MODE>(a, num_sms, st) : launch_own<MmaMath<FP8, 64, 1>, 64, MODE>(a, num_sms, st);
}

}  // namespace

long long own_rows(long long n_req, long long q_heads, int num_sms) {
    return n_req * q_heads + 2ll * num_sms * OWN_CTAS * OWN_WARPS * ATT_HEADS;
}

cudaError_t launch_attend_own(const AttendArgs &a, int num_sms, cudaStream_t st) {
    return a.kv.dtype == KV_E4M3 ? launch_own_type<true, SHARED>(a, num_sms, st) : launch_own_type<false, SHARED>(a, num_sms, st);
}
cudaError_t launch_attend_own_sinks(const AttendArgs &a, int num_sms, cudaStream_t st) { return launch_own_type<true, SINKS>(a, num_sms, st); }

}  // namespace scute
