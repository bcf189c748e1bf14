// One-token attention by warps on their own.  The batch's tiles (of a request's tokens;
// ROW_COST places for a request's start) are one sequence, cut into as many equal
// contiguous ranges as there are warps for each key/value head (and chunk of its query
// heads), in the same places for every head.  A warp takes a range of one head, fetches
// its keys and values into a ring of its own and leaves of each request in it a part
// (maximum, sum, unnormalised outputs) that launch_join (k_shared.cu) puts together with
// the other parts of the head.  Request r's part of range c is number r + c: no two of
// them are the same, without a count of the parts before.  The products are those of
// k_attend.cuh.
//
// What bounds it: memory, and for short rows the chain from a request's length over its
// pages to its first keys.  In k_attend.cuh a CTA's warps share every row, which ends with
// two of their barriers and a join in shared memory, about 3 us of its time; here a row's
// end is a warp's own and the others go on, and a warp's next rows are on their way while
// it computes this one.  Equal shares matter: with a row's tiles dealt out in items of
// equal length, two or three to a warp, SMs were at work 74 % of the time (200 requests,
// window 1000, 24 tokens before it, e4m3: 58.3 us, now 42.2).  Which launches come here,
// with both sides' times: serve.cu.  Behind shared beginnings (device time of the three
// launches in us, by CTAs and by warps): 64 requests 44.5 and 39.5, 250 of an e4m3 cache
// 73.8 and 60.9, 32 on a long document 113 and 110.
#include "k_attend.cuh"

namespace scute {

namespace {

// Eight warps on an SM, whose rings are three tiles: twelve with two tiles take 39.7 us behind
// 64 requests' shared beginning (39.0) and 58.8 to 59.1 behind the 250's (59.4).
constexpr int OWN_WARPS = 4;           // of a CTA
constexpr int OWN_CTAS = 2;            // of an SM, at most
constexpr int OWN_RING = 6;            // tiles of a warp's ring, at most
// What a request's start costs, in tiles: with 1 the 250 take 62.7 us, with 3 62.0.
constexpr int OWN_ROW_COST = 2;
// Of a range: with 6 the 64 requests take 40.8 us, with 10 43.6 (and the 32 116.5).
constexpr int LEAST_PLACES = 4;

// Tokens that a request sees, in tiles of positions first .. len - 1 (k_attend.cuh).
template <int MODE>
__device__ __forceinline__ int tiles_of(const AttendArgs &a, int r, int tt, Seen *y, bool *bad) {
    *y = seen_of<MODE>(a, r, tt, bad);
    return y->len > y->first ? (y->len - y->first + tt - 1) / tt : 0;
}

// Ranges of a head: one for each of its warps, two where there are too few warps to a head
// for even shares.
__host__ __device__ constexpr int own_ranges(int hz, int warps) {
    const int x = hz <= warps / 4 ? warps / hz : (int)(2ll * warps / hz);
    return x < 1 ? 1 : x;
}
// How the places are cut.
struct OwnCut {
    long long total;
    int ranges;
    __device__ __forceinline__ OwnCut(int places, int hz, int warps) {
        total = places;
        ranges = (int)min((long long)own_ranges(hz, warps), quotient(total + LEAST_PLACES - 1, LEAST_PLACES));
    }
    __device__ __forceinline__ int start(int c) const { return (int)quotient(total * c, ranges); }
    __device__ __forceinline__ int owner(int x) const { return (int)quotient((x + 1ll) * ranges - 1, total); }
};

// Walks the tiles of a warp's ranges: every `step`-th (range, head).
template <int MODE, int TT>
struct Cursor {
    const AttendArgs &a;
    const int *places_at;            // places of the requests before
    const OwnCut &cut;
    int hz, Z, step, item;
    int c, hk, z, begin, end;        // the range, its head and chunk, its places
    int r;                           // the piece: its request
    Seen seen;
    int pos, stop;                   // positions of the tile, and the piece's end

    __device__ __forceinline__ Cursor(const AttendArgs &args, const int *at, const OwnCut &of, int z_chunks, int warp, int warps)
        : a(args), places_at(at), cut(of), Z(z_chunks), step(warps), item(warp) {
        hz = a.kv.heads * Z;
        if (!more()) return;
        open();
        seek();
    }
    __device__ __forceinline__ bool more() const { return item < cut.ranges * hz; }
    __device__ __forceinline__ void open() {
        c = item / hz;
        hk = item - c * hz;
        z = hk % Z;
        hk /= Z;
        begin = cut.start(c);
        end = cut.start(c + 1);
        int hi = a.n_req - 1;                          // the last request whose places begin at `begin` or before
        for (r = 0; r < hi;) {
            const int mid = (r + hi + 1) >> 1;
            if (places_at[mid] <= begin) r = mid;
            else hi = mid - 1;
        }
    }
    // The first piece from request r on.
    __device__ __forceinline__ void seek() {
        for (;;) {
            for (; r < a.n_req && places_at[r] < end; ++r) {
                const int first = places_at[r] + OWN_ROW_COST, until = min(places_at[r + 1], end), t0 = max(0, begin - first);
                if (until <= first + t0) continue;     // only places of its start
                bool bad;
                tiles_of<MODE>(a, r, TT, &seen, &bad);
                pos = seen.first + t0 * TT;
                stop = min(seen.len, seen.first + (until - first) * TT);
                return;
            }
            item += step;
            if (!more()) return;
            open();
        }
    }
    __device__ __forceinline__ void next_piece() {
        ++r;
        seek();
    }
    __device__ __forceinline__ void next() {
        pos += TT;
        if (pos >= stop) next_piece();
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
    __shared__ int warp_sum[OWN_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.kv.dim, row_bytes = D * ESZ;
    uint8_t *const mine = smem + (size_t)warp * (ring * S::TILE + S::WARP_BYTES), *const extra = mine + ring * S::TILE;
    float *const s_m = reinterpret_cast<float *>(extra), *const s_l = s_m + HC;
    volatile unsigned *const s_ok = reinterpret_cast<unsigned *>(s_l + HC);
    int *const places_at = reinterpret_cast<int *>(smem + (size_t)OWN_WARPS * (ring * S::TILE + S::WARP_BYTES));
    const uint32_t ring_at = ptx::smem_u32(mine);
    // behind a head's elements every row of a tile stays zero
    if (row_bytes < ROW)
        for (int i = lane; i < ring * S::TILE / 16; i += 32) reinterpret_cast<uint4 *>(mine)[i] = make_uint4(0, 0, 0, 0);
    // (with shared beginnings the launch before is k_shared.cu's, which has waited for what
    // this one reads: only this one's end waits for it, for launch_join's sake)
    if constexpr (MODE != SHARED) ptx::grid_dep_wait();
    ptx::grid_dep_launch();

    // ------------------------------------------------ the plan: places of every request
    const int n = a.n_req, Z = (a.group + HC - 1) / HC, hz = a.kv.heads * Z, warps = gridDim.x * OWN_WARPS;
    const int per = (n + 32 * OWN_WARPS - 1) / (32 * OWN_WARPS), r0 = min(n, (int)threadIdx.x * per), r1 = min(n, r0 + per);
    bool any = false;
#pragma unroll 4
    for (int r = threadIdx.x; r < n; r += 32 * OWN_WARPS) {
        bool bad;
        Seen seen;
        const int tiles = tiles_of<MODE>(a, r, TT, &seen, &bad);
        places_at[r] = tiles ? tiles + OWN_ROW_COST : 0;
        any |= bad;
    }
    if (any && blockIdx.x == 0) atomicOr(a.status, STATUS_PAGES);
    __syncthreads();
    int sum = 0;
    for (int r = r0; r < r1; ++r) sum += places_at[r];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(ALL, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int at = inc - sum;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    for (int r = r0; r < r1; ++r) {
        const int x = places_at[r];
        places_at[r] = at;
        at += x;
    }
    if (r1 == n && r0 < n) places_at[n] = at;
    __syncthreads();
    const OwnCut cut(places_at[n], hz, warps);
    for (int r = blockIdx.x * 32 * OWN_WARPS + threadIdx.x; r < n; r += gridDim.x * 32 * OWN_WARPS) {
        const int x = places_at[r] + OWN_ROW_COST, y = places_at[r + 1];
        const int first = x < y ? cut.owner(x) : 0;
        a.own_at[r] = make_int2(r + first, x < y ? cut.owner(y - 1) - first + 1 : 0);
    }

    // ------------------------------------------------ the warp's items
    constexpr int LR = ROW >= 512 ? 32 : ROW / 16, RI = 32 / LR, SUB = TT < 16 ? TT : 16;
    static_assert(ROW < 512, "a row is an instruction's part");
    const int piece = lane % LR, row0 = lane / LR;
    const bool here = piece * 16 < row_bytes;
    const long long tok_bytes = a.kv.token_stride * ESZ;
    const uint32_t lane_at = place_of<ROW>(row0, piece);
    const uint64_t policy = ptx::make_policy_evict_first();
    const int gw = blockIdx.x * OWN_WARPS + warp;
    Cursor<MODE, TT> f(a, places_at, cut, Z, gw, warps);       // the tile to be fetched
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
    Cursor<MODE, TT> w(a, places_at, cut, Z, gw, warps);       // the tile to be computed
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
        const long long part_row = (long long)(w.r + w.c) * a.q_heads + h0;
        const float scale = (a.kv.k_scale ? a.kv.k_scale[w.hk] : 1.f) * a.scale;
        math.queries(ahead, a.softcap > 0.f ? scale : scale * LOG2E);
        const int last = (w.stop - w.pos + TT - 1) / TT;
        w.next_piece();
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
int heads_of(int group) { return group > 8 ? 16 : 8; }           // of a chunk
template <bool FP8, int MODE>
cudaError_t launch_own_type(const AttendArgs &a, int num_sms, cudaStream_t st) {
    const bool wide = heads_of(a.group) > 8;
    if (a.kv.dim > 64)
        return wide ? launch_own<MmaMath<FP8, 128, 2>, 128, MODE>(a, num_sms, st) : launch_own<MmaMath<FP8, 128, 1>, 128, MODE>(a, num_sms, st);
    return wide ? launch_own<MmaMath<FP8, 64, 2>, 64, MODE>(a, num_sms, st) : launch_own<MmaMath<FP8, 64, 1>, 64, MODE>(a, num_sms, st);
}

}  // namespace

// (with one CTA on an SM there are no more ranges than with two)
long long own_rows(long long n_req, int q_heads, int kv_heads, int num_sms) {
    const int group = q_heads / kv_heads, hc = heads_of(group);
    return (n_req + own_ranges(kv_heads * ((group + hc - 1) / hc), num_sms * OWN_CTAS * OWN_WARPS)) * q_heads;
}

cudaError_t launch_attend_own(const AttendArgs &a, int num_sms, cudaStream_t st) {
    return a.kv.dtype == KV_E4M3 ? launch_own_type<true, SHARED>(a, num_sms, st) : launch_own_type<false, SHARED>(a, num_sms, st);
}
cudaError_t launch_attend_own_sinks(const AttendArgs &a, int num_sms, cudaStream_t st) {
    return a.kv.dtype == KV_E4M3 ? launch_own_type<true, SINKS>(a, num_sms, st) : launch_own_type<false, SINKS>(a, num_sms, st);
}

}  // namespace scute
