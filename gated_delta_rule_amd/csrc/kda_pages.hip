// Pages of a cache (gfx950): new tokens into them, and which slot holds which.
// Semantics: include/kda_attn.h (append) and include/kda_pages.h.
//
// Who gets which page depends on everyone before, so one workgroup of 16
// waves decides: prefix sums of what the slots need, then the free pages in
// order of their numbers, 16384 counts at a time, until there are enough.  Its
// time is that of a handful of reads in sequence.
// Everything that needs no order (table rows, counts, the data of pages) runs
// on the whole GPU in the launches behind it.  Counts of holders are changed
// by integer atomics, whose order does not change the sum.
//   Moving 0.68 GB of pages together (written once, read once): 11 us to plan,
// 270 to move, 5.0 TB/s; forking 224 slots of 32 requests with 4 layers' open
// pages: 12 to plan, 6 to count, 36 to copy.
#include "kda_attn_tile.h"

namespace kda {

// ----------------------------------------------------------------- append

template <typename InT>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendParams p) {
    constexpr int EV = 16 / (int)sizeof(InT);
    const int per = p.G * p.D / EV;                   // pieces of a token row
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / per;
    if (row >= p.rows) return;
    const int c = (int)(i - row * per) * EV, g = c / p.D, d = c - g * p.D;
    int n;
    AttnRange r;
    if (!p.cu) {
        n = (int)(row / p.T);
        r = AttnRange{n * p.T, n * p.T + p.T};
    } else {
        int lo = 0, hi = p.n_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (attn_range(p.cu, p.rows, p.T, mid).start <= row) lo = mid;
            else hi = mid;
        }
        n = lo;
        r = attn_range(p.cu, p.rows, p.T, n);
        if (row < r.start || row >= r.end) return;
    }
    const int64_t most = (int64_t)p.max_pages << p.page_shift;
    int64_t len = p.lengths[n];
    len = len < 0 ? 0 : len < most ? len : most;
    const int64_t x = len - (r.end - row);
    if (x < 0) return;
    const int32_t page = p.table[(int64_t)n * p.max_pages + (x >> p.page_shift)];
    if (page < 0 || page >= p.n_pages) return;
    const int64_t to = page * p.page_stride + (((int64_t)g << p.page_shift) + (x & ((1 << p.page_shift) - 1))) * p.D + d;
    *reinterpret_cast<u32x4*>((InT*)p.k_pages + to) = *reinterpret_cast<const u32x4*>((const InT*)p.k + row * p.k_stride + c);
    *reinterpret_cast<u32x4*>((InT*)p.v_pages + to) = *reinterpret_cast<const u32x4*>((const InT*)p.v + row * p.v_stride + c);
}

hipError_t launch_kv_append(const AppendParams& p, bool bf16_in, hipStream_t stream) {
    const int64_t pieces = p.rows * p.G * p.D / (bf16_in ? 8 : 4);
    if (pieces == 0) return hipSuccess;
    const dim3 grid((uint32_t)((pieces + 255) / 256));
    if (bf16_in) kv_append_kernel<__bf16><<<grid, 256, 0, stream>>>(p);
    else kv_append_kernel<float><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
}

// ------------------------------------------------------- one workgroup's part

constexpr int PG_THREADS = 1024, PG_WAVES = PG_THREADS / 64, PG_EACH = 16;   // EACH: counts per thread and step
constexpr int PG_STEP = PG_THREADS * PG_EACH;

// Sum of x over the threads before this one; `total` over all.  s: PG_WAVES + 1 ints.
__device__ __forceinline__ int32_t block_before(int32_t x, int32_t* s, int32_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t up = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t y = __shfl_up(up, d);
        if (lane >= d) up += y;
    }
    __syncthreads();   // (s of the call before has been read)
    if (lane == 63) s[wave] = up;
    __syncthreads();
    int32_t base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < PG_WAVES; ++w) {
        if (w < wave) base += s[w];
        total += s[w];
    }
    return base + up - x;
}
// What this workgroup's atomics and writes have left in L2, where they are done
// once a barrier has been passed (past the compute unit's own cache, which
// atomics do not go through).
__device__ __forceinline__ int32_t fresh_load(const int32_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Which of the pages base + e * PG_THREADS + thread are free, as bits e.
__device__ __forceinline__ uint32_t free_bits(const int32_t* refs, int64_t base, int32_t n_pages) {
    uint32_t m = 0;
    int32_t r[PG_EACH];
#pragma unroll
    for (int e = 0; e < PG_EACH; ++e) {
        const int64_t at = base + e * PG_THREADS + threadIdx.x;
        r[e] = at < n_pages ? fresh_load(refs + at) : 1;
    }
#pragma unroll
    for (int e = 0; e < PG_EACH; ++e) m |= (r[e] <= 0 ? 1u : 0u) << e;
    return m;
}
// Calls put(e, rank) for the bits e that are set, ranked in the order of
// e * PG_THREADS + thread over the workgroup; returns how many there are.
// s: PG_EACH * PG_WAVES ints.
template <typename F>
__device__ __forceinline__ int32_t in_order(uint32_t bits, int32_t* s, F put) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    static_assert(PG_EACH == 16 && PG_WAVES == 16, "four counts per lane");
    uint64_t b[PG_EACH];
    __syncthreads();   // (s has been read)
#pragma unroll
    for (int e = 0; e < PG_EACH; ++e) {
        b[e] = __ballot(bits >> e & 1);
        if (lane == e) s[e * PG_WAVES + wave] = __popcll(b[e]);
    }
    __syncthreads();
    int32_t c[4], mine = 0, up;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] = s[4 * lane + i];
        mine += c[i];
    }
    up = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t y = __shfl_up(up, d);
        if (lane >= d) up += y;
    }
    int32_t before = up - mine;   // this lane's four counts belong to waves 4 (lane & 3) .. + 3 of one e
#pragma unroll
    for (int i = 0; i < 3; ++i) before += i < (wave & 3) ? c[i] : 0;
#pragma unroll
    for (int e = 0; e < PG_EACH; ++e) {
        const int32_t first = __builtin_amdgcn_readlane(before, 4 * e + (wave >> 2));
        if (bits >> e & 1) put(e, first + (int32_t)__popcll(b[e] & ((1ull << lane) - 1)));
    }
    return __builtin_amdgcn_readlane(up, 63);
}
// Free pages, counted up to `enough`; bits: of the first step.
__device__ __forceinline__ int64_t count_free(const int32_t* refs, int32_t n_pages, int64_t enough, int32_t* s, uint32_t& bits) {
    int64_t found = 0;
    for (int64_t base = 0; base < n_pages && found < enough; base += PG_STEP) {
        const uint32_t m = free_bits(refs, base, n_pages);
        if (base == 0) bits = m;
        int32_t total;
        block_before(__popc(m), s, total);
        found += total;
    }
    return found;
}
// Gives out `count` free pages in order: put(rank, page) for rank < count.
// The pages become held once, in refs and in `bits` (of the first step), so
// that the next call goes on behind them.
template <typename F>
__device__ __forceinline__ void give_out(int32_t* refs, int32_t n_pages, int32_t count, int32_t* s, uint32_t& bits, F put) {
    int32_t done = 0;
    for (int64_t base = 0; base < n_pages && done < count; base += PG_STEP) {
        const uint32_t m = base == 0 ? bits : free_bits(refs, base, n_pages);
        done += in_order(m, s, [&](int e, int32_t rank) {
            if (done + rank >= count) return;
            const int32_t page = (int32_t)(base + e * PG_THREADS + threadIdx.x);
            refs[page] = 1;
            if (base == 0) bits &= ~(1u << e);
            put(done + rank, page);
        });
    }
}
__device__ __forceinline__ int32_t pages_of(int32_t len, int shift) {
    return (int32_t)(((int64_t)len + (1 << shift) - 1) >> shift);
}
__device__ __forceinline__ int32_t clamp_length(int32_t len, const PagesParams& p) {
    const int64_t most = (int64_t)p.max_pages << p.page_shift;
    return len < 0 ? 0 : (int32_t)(len < most ? len : most);
}
// Largest i with off[i] <= rank, off ascending.
__device__ __forceinline__ int owner_of(const int32_t* off, int n, int32_t rank) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= rank) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ----------------------------------------------------------------- resize

__global__ __launch_bounds__(PG_THREADS) void kv_resize_kernel(PagesParams p) {
    __shared__ int32_t s[PG_EACH * PG_WAVES], off[PG_THREADS], from[PG_THREADS];
    const int tid = threadIdx.x;
    int32_t* refs = p.refs_out;
    int64_t need_all = 0;
    for (int s0 = 0; s0 < p.n_slots; s0 += PG_THREADS) {   // what is needed, and what is given up
        const int slot = s0 + tid;
        int32_t d = 0, after = 0;
        if (slot < p.n_slots) {
            after = pages_of(clamp_length(p.want[slot], p), p.page_shift);
            d = after - pages_of(clamp_length(p.lengths[slot], p), p.page_shift);
        }
        int32_t total, gone;
        block_before(d > 0 ? d : 0, s, total);   // (table entries: below 2^31 in all)
        need_all += total;
        off[tid] = block_before(d < 0 ? -d : 0, s, gone);
        from[tid] = after;
        __syncthreads();
        for (int32_t i = tid; i < gone; i += PG_THREADS) {
            const int o = owner_of(off, PG_THREADS, i);
            int32_t* entry = p.table_out + (int64_t)(s0 + o) * p.max_pages + from[o] + i - off[o];
            const int32_t page = *entry;
            if (page >= 0 && page < p.n_pages) atomicSub(refs + page, 1);
            *entry = -1;
        }
        __syncthreads();
    }
    uint32_t bits = 0;
    const int64_t n_free = need_all > 0 ? count_free(refs, p.n_pages, need_all, s, bits) : 0;
    int64_t upto = 0;
    for (int s0 = 0; s0 < p.n_slots; s0 += PG_THREADS) {
        const int slot = s0 + tid;
        int32_t need = 0, want = 0, len = 0, before = 0;
        if (slot < p.n_slots) {
            want = clamp_length(p.want[slot], p);
            len = clamp_length(p.lengths[slot], p);
            before = pages_of(len, p.page_shift);
            const int32_t d = pages_of(want, p.page_shift) - before;
            need = d > 0 ? d : 0;
        }
        bool ok = true;
        if (need_all > 0) {
            int32_t total, served;
            const int64_t at = upto + block_before(need, s, total);
            ok = need == 0 || at + need <= n_free;
            upto += total;
            off[tid] = block_before(ok ? need : 0, s, served);
            from[tid] = before;
            __syncthreads();
            // (slots without a need share the next one's offset: the last of equal ones has the page)
            give_out(refs, p.n_pages, served, s, bits, [&](int32_t rank, int32_t page) {
                const int i = owner_of(off, PG_THREADS, rank);
                p.table_out[(int64_t)(s0 + i) * p.max_pages + from[i] + rank - off[i]] = page;
            });
            __syncthreads();
        }
        if (slot < p.n_slots) {
            p.lengths_out[slot] = ok ? want : len;
            if (p.ok) p.ok[slot] = ok;
        }
    }
}

hipError_t launch_kv_resize(const PagesParams& p, hipStream_t stream) {
    kv_resize_kernel<<<1, PG_THREADS, 0, stream>>>(p);
    return hipGetLastError();
}

// ------------------------------------------------------------------- fork

constexpr int FORK_NEAR = 8192;   // slots

// Workspace: the first pair of each destination [n_slots], then per pair: what follows, then rows [n, max_pages].
struct ForkPlan {
    int32_t go;        // the pair is carried out
    int32_t length;    // of the source
    int32_t cols;      // entries of the destination's row that change
    int32_t from, to;  // page to copy and its copy, or -1
};
__device__ __forceinline__ ForkPlan* fork_plans(const PagesParams& p) { return (ForkPlan*)(p.ws + ((p.n_slots + 3) & ~3)); }
__device__ __forceinline__ int32_t* fork_rows(const PagesParams& p) {
    return p.ws + (((int64_t)p.n_slots + 3) & ~3) + (int64_t)p.n * (sizeof(ForkPlan) / 4);
}

// Entry col of pair i: the counts, and the new row into the workspace (a source
// may be another pair's destination).
__device__ __forceinline__ void fork_count(const PagesParams& p, int64_t i, int32_t col) {
    const ForkPlan f = fork_plans(p)[i];
    if (!f.go || col >= f.cols) return;
    const int32_t used = pages_of(f.length, p.page_shift), old = pages_of(clamp_length(p.lengths[p.dst[i]], p), p.page_shift);
    int32_t page = -1;
    if (col < used) {
        page = p.table[(int64_t)p.src[i] * p.max_pages + col];
        if (f.to >= 0 && col == used - 1) page = f.to;   // (its count is one already)
        else if (page >= 0 && page < p.n_pages) atomicAdd(p.refs_out + page, 1);
    }
    if (col < old) {
        const int32_t had = p.table[(int64_t)p.dst[i] * p.max_pages + col];
        if (had >= 0 && had < p.n_pages) atomicSub(p.refs_out + had, 1);
    }
    fork_rows(p)[i * p.max_pages + col] = page;
}

__global__ __launch_bounds__(PG_THREADS) void kv_fork_plan_kernel(PagesParams p, bool count) {
    __shared__ int32_t s[PG_EACH * PG_WAVES], off[PG_THREADS];
    const int tid = threadIdx.x;
    int32_t* refs = p.refs_out;
    ForkPlan* plan = fork_plans(p);
    // the first pair of each destination, in LDS if it has room
    __shared__ int32_t near[FORK_NEAR];
    const bool in_lds = p.n_slots <= FORK_NEAR;
    for (int i = tid; i < p.n_slots; i += PG_THREADS) (in_lds ? near : p.ws)[i] = INT32_MAX;
    __syncthreads();
    for (int i = tid; i < p.n; i += PG_THREADS) {
        const int32_t d = p.dst[i];
        if (d >= 0 && d < p.n_slots) {
            if (in_lds) atomicMin(near + d, i);
            else atomicMin(p.ws + d, i);
        }
    }
    __syncthreads();
    int64_t need_all = 0;
    for (int i0 = 0; i0 < p.n; i0 += PG_THREADS) {
        const int i = i0 + tid;
        ForkPlan f = {0, 0, 0, -1, -1};
        if (i < p.n) {
            const int32_t a = p.src[i], d = p.dst[i];
            if (a >= 0 && a < p.n_slots && d >= 0 && d < p.n_slots && (in_lds ? near[d] : fresh_load(p.ws + d)) == i) {
                f.go = 1;
                f.length = clamp_length(p.lengths[a], p);
                const int32_t used = pages_of(f.length, p.page_shift), old = pages_of(clamp_length(p.lengths[d], p), p.page_shift);
                f.cols = a == d ? 0 : used > old ? used : old;
                if (a != d && (f.length & ((1 << p.page_shift) - 1))) {
                    const int32_t page = p.table[(int64_t)a * p.max_pages + used - 1];
                    if (page >= 0 && page < p.n_pages) f.from = page;
                }
            }
            plan[i] = f;
        }
        int32_t total;
        block_before(f.from >= 0, s, total);
        need_all += total;
    }
    uint32_t bits = 0;
    const int64_t n_free = need_all > 0 ? count_free(refs, p.n_pages, need_all, s, bits) : 0;
    int64_t upto = 0;
    for (int i0 = 0; i0 < p.n; i0 += PG_THREADS) {
        const int i = i0 + tid;
        ForkPlan f = {0, 0, 0, -1, -1};
        if (i < p.n) f = plan[i];   // (written by this thread)
        const int32_t need = f.from >= 0;
        int32_t total, served;
        const int64_t at = upto + block_before(need, s, total);
        const bool ok = f.go && (need == 0 || at + need <= n_free);
        upto += total;
        off[tid] = block_before(ok ? need : 0, s, served);
        if (!ok || !need) f.from = -1;
        if (f.go && !ok) f.go = f.cols = 0;
        if (i < p.n) {
            plan[i] = f;
            if (p.ok) p.ok[i] = ok;
        }
        __syncthreads();
        if (served > 0) {
            give_out(refs, p.n_pages, served, s, bits, [&](int32_t rank, int32_t page) {
                plan[i0 + owner_of(off, PG_THREADS, rank)].to = page;
            });
            __syncthreads();
        }
        __syncthreads();
    }
    if (!count) return;
    const int32_t entries = p.n * p.max_pages;
    for (int32_t k = tid; k < entries; k += PG_THREADS) {
        const int32_t i = k / p.max_pages;
        fork_count(p, i, k - i * p.max_pages);
    }
}

__global__ __launch_bounds__(256) void kv_fork_count_kernel(PagesParams p, int32_t chunks) {
    const int64_t i = blockIdx.x / (uint32_t)chunks;
    fork_count(p, i, (int32_t)(blockIdx.x % (uint32_t)chunks) * 256 + threadIdx.x);
}

// Bytes [piece * 16 KB, ...) of a page, all tensors in line.
constexpr int kCopyLoads = 4;
constexpr int64_t kCopyPiece = kCopyLoads * 4096;
__device__ __forceinline__ void copy_piece(const PageData& d, int64_t from, int64_t to, int64_t piece) {
    for (int t = 0; t < d.n; ++t) {
        const int64_t pieces = (d.bytes[t] + kCopyPiece - 1) / kCopyPiece;
        if (piece >= pieces) {
            piece -= pieces;
            continue;
        }
        const char* a = d.base[t] + from * d.stride[t] + piece * kCopyPiece;
        char* b = d.base[t] + to * d.stride[t] + piece * kCopyPiece;
        const int32_t at = threadIdx.x * 16;
        if ((piece + 1) * kCopyPiece <= d.bytes[t]) {
            u32x4 r[kCopyLoads];
#pragma unroll
            for (int k = 0; k < kCopyLoads; ++k) r[k] = *reinterpret_cast<const u32x4*>(a + at + k * 4096);
#pragma unroll
            for (int k = 0; k < kCopyLoads; ++k) *reinterpret_cast<u32x4*>(b + at + k * 4096) = r[k];
        } else {
            const int32_t left = (int32_t)(d.bytes[t] - piece * kCopyPiece);
            for (int32_t i = at; i < left; i += 4096) *reinterpret_cast<u32x4*>(b + i) = *reinterpret_cast<const u32x4*>(a + i);
        }
        return;
    }
}
static int64_t copy_pieces(const PageData& d) {
    int64_t n = 0;
    for (int t = 0; t < d.n; ++t) n += (d.bytes[t] + kCopyPiece - 1) / kCopyPiece;
    return n;
}

// The rows from the workspace, and the copies' data.
__global__ __launch_bounds__(256) void kv_fork_write_kernel(PagesParams p, int32_t chunks, int32_t walkers, int64_t pieces) {
    const uint32_t per = (uint32_t)(chunks + walkers);
    const int64_t i = blockIdx.x / per;
    const int32_t w = (int32_t)(blockIdx.x % per);
    const ForkPlan f = fork_plans(p)[i];
    if (!f.go) return;
    if (w < chunks) {
        const int32_t col = w * 256 + threadIdx.x, d = p.dst[i];
        if (col < f.cols) p.table_out[(int64_t)d * p.max_pages + col] = fork_rows(p)[i * p.max_pages + col];
        if (w == 0 && threadIdx.x == 0 && p.src[i] != d) p.lengths_out[d] = f.length;
        return;
    }
    if (f.to < 0) return;
    for (int64_t k = w - chunks; k < pieces; k += walkers) copy_piece(p.data, f.from, f.to, k);
}

hipError_t launch_kv_fork(const PagesParams& p, hipStream_t stream) {
    // Few entries are counted by the planning workgroup, more of them by a launch
    // of their own (2.5 us on the host, 2 to 4 on the GPU): 16 rounds of the
    // workgroup take about as long.
    const bool count = (int64_t)p.n * p.max_pages <= 16 * PG_THREADS;
    kv_fork_plan_kernel<<<1, PG_THREADS, 0, stream>>>(p, count);
    const int32_t chunks = (p.max_pages + 255) / 256;
    if (chunks > 0) {   // (max_pages 0: lengths are 0, and stay so)
        if (!count) kv_fork_count_kernel<<<dim3((uint32_t)p.n * chunks), 256, 0, stream>>>(p, chunks);
        const int64_t pieces = copy_pieces(p.data);
        const int32_t walkers = (int32_t)(pieces < 64 ? pieces : 64);
        kv_fork_write_kernel<<<dim3((uint32_t)p.n * (uint32_t)(chunks + walkers)), 256, 0, stream>>>(p, chunks, walkers, pieces);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------- compact

// Workspace: moves, pad; then [n_pages] each: pages that move, pages that
// receive them, and the rank of each page that moves (-1: it stays).
__global__ __launch_bounds__(PG_THREADS) void kv_compact_plan_kernel(PagesParams p) {
    __shared__ int32_t s[PG_EACH * PG_WAVES];
    const int32_t N = p.n_pages;
    uint32_t bits = 0;
    const int32_t n_live = N - (int32_t)count_free(p.refs, N, (int64_t)N + 1, s, bits);
    int32_t *mov = p.ws + 4, *hol = mov + N, *rank_of = hol + N;
    int32_t moved = 0, holes = 0;
    for (int64_t base = 0; base < N; base += PG_STEP) {
        const uint32_t free = base == 0 ? bits : free_bits(p.refs, base, N);
        uint32_t below = 0, exist = 0;   // pages < n_live, pages < N
#pragma unroll
        for (int e = 0; e < PG_EACH; ++e) {
            const int64_t at = base + e * PG_THREADS + threadIdx.x;
            below |= (at < n_live ? 1u : 0u) << e;
            exist |= (at < N ? 1u : 0u) << e;
            if (at < N && (at < n_live || free >> e & 1)) rank_of[at] = -1;   // (stays)
        }
        const int64_t mine = base + threadIdx.x;
        if (base + PG_STEP > n_live)
            moved += in_order(~free & exist & ~below, s, [&](int e, int32_t rank) {
                mov[moved + rank] = (int32_t)(mine + e * PG_THREADS);
                rank_of[mine + e * PG_THREADS] = moved + rank;
            });
        if (base < n_live)
            holes += in_order(free & below, s, [&](int e, int32_t rank) { hol[holes + rank] = (int32_t)(mine + e * PG_THREADS); });
    }
    if (threadIdx.x == 0) {
        p.ws[0] = moved;
        p.n_live[0] = n_live;
    }
}

__global__ __launch_bounds__(256) void kv_compact_write_kernel(PagesParams p, int32_t copiers, int64_t pieces) {
    const int32_t N = p.n_pages, moves = p.ws[0], n_live = p.n_live[0];
    const int32_t *mov = p.ws + 4, *hol = mov + N, *rank_of = hol + N;
    if ((int32_t)blockIdx.x < copiers) {
        for (int64_t k = blockIdx.x; k < moves * pieces; k += copiers) {
            const int64_t m = k / pieces;
            copy_piece(p.data, mov[m], hol[m], k - m * pieces);
        }
        return;
    }
    const int64_t step = (int64_t)(gridDim.x - copiers) * 256, me = (int64_t)(blockIdx.x - copiers) * 256 + threadIdx.x;
    const bool in_place = p.refs_out == p.refs;
    for (int64_t i = me; i < N; i += step) {
        if (i < moves) {
            const int32_t r = p.refs[mov[i]];
            p.refs_out[hol[i]] = r;
            p.refs_out[mov[i]] = 0;
        }
        // pages that neither move nor receive one
        if (!in_place && rank_of[i] < 0 && !(i < n_live && p.refs[i] <= 0)) p.refs_out[i] = p.refs[i];
    }
    const int64_t entries = (int64_t)p.n_slots * p.max_pages;
    for (int64_t i = me; i < entries; i += step) {
        const int32_t slot = (int32_t)(i / p.max_pages), col = (int32_t)(i - (int64_t)slot * p.max_pages);
        int32_t page = -1;
        if (col < pages_of(clamp_length(p.lengths[slot], p), p.page_shift)) {
            page = p.table[i];
            if (page >= 0 && page < N && rank_of[page] >= 0) page = hol[rank_of[page]];
        }
        p.table_out[i] = page;
    }
}

hipError_t launch_kv_compact(const PagesParams& p, hipStream_t stream) {
    kv_compact_plan_kernel<<<1, PG_THREADS, 0, stream>>>(p);
    const int64_t pieces = copy_pieces(p.data);
    const int64_t all = (int64_t)p.n_pages * pieces, entries = (int64_t)p.n_slots * p.max_pages;
    const int32_t copiers = (int32_t)(all < 2048 ? all : 2048);
    const int64_t work = entries > p.n_pages ? entries : p.n_pages;
    const int32_t rest = (int32_t)((work + 255) / 256 < 512 ? (work + 255) / 256 : 512);
    if (copiers + rest > 0) kv_compact_write_kernel<<<dim3((uint32_t)(copiers + rest)), 256, 0, stream>>>(p, copiers, pieces);
    return hipGetLastError();
}

}  // namespace kda
