// Vector-state gated linear recurrence, forward and backward, in one pass over the data.
//
// h_t = a_t h_{t-1} + x_t with a_t = exp(g_t) is a chain of affine maps, and maps compose: rows r..s together take
// the entering state h to A h + H, with A the product of their decays and H the state they reach from zero.  So the
// time axis is cut: a thread folds RPT consecutive rows of two channels into (A, H), the CTA composes its warps'
// maps, a cluster of S CTAs composes its CTAs' maps through distributed shared memory, and the state entering every
// thread's rows follows; the thread then runs its rows again from that state (decays kept in registers, inputs still
// in shared memory) and writes them.  The cluster walks the sequence S * R rows at a time and carries the state.
// The backward is the same chain from the last row to the first: mu_t = a_t (dh_t + mu_{t+1}).
//
// Every input is read once and every output written once.  The order of all sums is fixed by the shape.
#include <algorithm>
#include <type_traits>

#include "api_common.h"
#include "gla_internal.h"
#include "layer_internal.h"
#include "tc_ptx.cuh"

namespace gla {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kCols = 64;       // channels of a CTA: two per lane
constexpr int kMaxCluster = 8;
constexpr int kSlots = 2;       // tiles whose maps are in shared memory at a time

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank)   // the same variable of another CTA
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(p)), "r"(rank));
    return r;
}

// 16 bytes of global memory to shared memory, the first `bytes` of them read and the rest zeros.
__device__ __forceinline__ void copy16(void *dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Rows [begin, begin + len) of sequence n; false (and a status) where the offsets are bad.
__device__ __forceinline__ bool sequence_rows(const ScanArgs &a, int n, int64_t &begin, int &len)
{
    if (!a.cu) {
        begin = (int64_t)n * a.T;
        len = a.T;
        return true;
    }
    const int lo = a.cu[n], hi = a.cu[n + 1];
    const bool ok = lo >= 0 && hi >= lo && hi <= a.T && (n > 0 || lo == 0) && (n < a.N - 1 || hi == a.T);
    if (!ok && threadIdx.x == 0)
        report(a.status, GLA_ERR_INVALID_ARG);
    begin = lo;
    len = hi - lo;
    return ok;
}

// Two adjacent 16-bit values in a word.
template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t w);
template <>
__device__ __forceinline__ float2 widen2<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 widen2<__half>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t narrow2(float2 v);
template <>
__device__ __forceinline__ uint32_t narrow2<__nv_bfloat16>(float2 v)
{
    const __nv_bfloat162 b = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t *>(&b);
}
template <>
__device__ __forceinline__ uint32_t narrow2<__half>(float2 v)
{
    const __half2 b = __float22half2_rn(v);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// One R x kCols tile of a row-strided tensor in shared memory.  Rows whose bytes start and step in 16-byte units
// (ALIGNED) lie as they are; others are copied from the 16-byte unit that holds their first byte, so every row has a
// shift of its own.
template <typename T, int R, bool ALIGNED>
struct Tile {
    static constexpr int kUnits = kCols * (int)sizeof(T) / 16 + (ALIGNED ? 0 : 1);
    static constexpr int kPitch = kUnits * 16;
    static constexpr int kBytes = R * kPitch;

    // Row j of the tile is row r0 + DIR j of the sequence (src: its first row at the tile's first channel); rows
    // outside [0, len) and channels from `cols` on are zeros.  A thread copies one 16-byte column of the tile.
    template <int DIR>
    static __device__ __forceinline__ void load(char *dst, const T *src, int64_t ld, int r0, int len, int cols)
    {
        const int width = min(kCols, cols) * (int)sizeof(T);
        if constexpr (ALIGNED) {
            constexpr int kStep = kThreads / kUnits;   // rows between a thread's copies
            const int u = threadIdx.x % kUnits, j0 = threadIdx.x / kUnits;
            const bool in = 16 * u < width;
            const T *p = src + (int64_t)(r0 + DIR * j0) * ld + 16 / (int)sizeof(T) * u;
            char *q = dst + j0 * kPitch + 16 * u;
            if (width == kPitch && (unsigned)r0 < (unsigned)len && (unsigned)(r0 + DIR * (R - 1)) < (unsigned)len) {
#pragma unroll
                for (int j = 0; j < R; j += kStep)
                    copy16(q + j * kPitch, p + DIR * (int64_t)j * ld);
                return;
            }
#pragma unroll
            for (int j = 0; j < R; j += kStep) {
                const int r = r0 + DIR * (j0 + j);
                const bool ok = in && (unsigned)r < (unsigned)len;
                copy16(q, ok ? p : src, ok ? 16 : 0);
                p += DIR * kStep * ld;
                q += kStep * kPitch;
            }
        } else {
            for (int i = threadIdx.x; i < R * kUnits; i += kThreads) {
                const int j = i / kUnits, u = i - j * kUnits, r = r0 + DIR * j;
                const bool ok = (unsigned)r < (unsigned)len;
                const T *p = src + (ok ? r * ld : 0);
                const int shift = (int)(reinterpret_cast<uintptr_t>(p) & 15);
                const int bytes = ok ? max(0, min(16, shift + width - 16 * u)) : 0;
                const char *from = reinterpret_cast<const char *>(p) - shift;
                copy16(dst + j * kPitch + 16 * u, from + (bytes ? 16 * u : 0), bytes);
            }
        }
    }

    // The lane's two channels of row j (row r of the sequence): 2 l and 2 l + 1, or l and l + 32 where rows are shifted.
    static __device__ __forceinline__ float2 read(const char *tile, int j, const T *src, int64_t ld, int r)
    {
        const int lane = threadIdx.x & 31;
        const char *row = tile + j * kPitch;
        if constexpr (ALIGNED) {
            if constexpr (sizeof(T) == 4)
                return *reinterpret_cast<const float2 *>(row + 8 * lane);
            else
                return widen2<T>(*reinterpret_cast<const uint32_t *>(row + 4 * lane));
        } else {
            // only the low bits of the address count (rows outside the sequence are zeros at any shift)
            const uint32_t at = (uint32_t)reinterpret_cast<uintptr_t>(src) + (uint32_t)r * (uint32_t)ld * (uint32_t)sizeof(T);
            const T *p = reinterpret_cast<const T *>(row + (at & 15));
            return make_float2(widen(p[lane]), widen(p[lane + 32]));
        }
    }
};

// The lane's two channels, and the stores of a pair.
template <bool ALIGNED>
struct Pair {
    int d[2];
    bool on[2];
    __device__ __forceinline__ Pair(int d0, int D)
    {
        const int lane = threadIdx.x & 31;
        d[0] = d0 + (ALIGNED ? 2 * lane : lane);
        d[1] = d0 + (ALIGNED ? 2 * lane + 1 : lane + 32);
        on[0] = d[0] < D;
        on[1] = d[1] < D;
    }
    template <bool WHOLE, typename T>   // WHOLE: both channels exist
    __device__ __forceinline__ void store(T *row, float2 v) const
    {
        if constexpr (ALIGNED) {
            if (!WHOLE && !on[0])
                return;
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<float2 *>(row + d[0]) = v;
            else
                *reinterpret_cast<uint32_t *>(row + d[0]) = narrow2<T>(v);
        } else {
            if (WHOLE || on[0])
                row[d[0]] = narrow<T>(v.x);
            if (WHOLE || on[1])
                row[d[1]] = narrow<T>(v.y);
        }
    }
    __device__ __forceinline__ float2 state(const float *p, int64_t at) const   // p[at + d] or zeros
    {
        return make_float2(p && on[0] ? p[at + d[0]] : 0.f, p && on[1] ? p[at + d[1]] : 0.f);
    }
    __device__ __forceinline__ void put_state(float *p, int64_t at, float2 v) const
    {
        if (on[0])
            p[at + d[0]] = v.x;
        if (on[1])
            p[at + d[1]] = v.y;
    }
};

// Two channels at a time: one instruction for both (the same roundings as one by one).
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 decay2(float2 g) { return make_float2(decay(g.x), decay(g.y)); }

// An affine map h -> A h + H of a lane's two channels.
struct Map {
    float2 A, H;
    __device__ __forceinline__ Map() : A{1.f, 1.f}, H{0.f, 0.f} {}
    __device__ __forceinline__ Map(float4 v) : A{v.x, v.y}, H{v.z, v.w} {}
    __device__ __forceinline__ float4 packed() const { return make_float4(A.x, A.y, H.x, H.y); }
    __device__ __forceinline__ void then(const Map &m)   // this map, then m
    {
        A = mul2(A, m.A);
        H = fma2(m.A, H, m.H);
    }
    __device__ __forceinline__ float2 operator()(float2 h) const { return fma2(A, h, H); }
};

struct Shared {
    float4 warps[kSlots][kWarps][32];       // the maps of a tile's warps
    float4 ctas[kSlots][kMaxCluster][32];   // the maps of the cluster's CTAs, pushed by each of them
    uint64_t full[kSlots];                  // all CTAs' maps of the slot's tile are here
    int abort;
};

__device__ __forceinline__ void open_cluster(Shared &sh)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i)
            tc::bar_init(&sh.full[i], 1);
        sh.abort = 0;
        tc::bar_fence_init();
    }
    __syncthreads();
    cluster_sync();   // every CTA's barriers are set up
}
__device__ __forceinline__ void close_cluster(Shared &sh, int *status)
{
    cluster_sync();   // nobody leaves while another may push into it
    if (threadIdx.x == 0 && sh.abort)
        report(status, GLA_ERR_TIMEOUT);
}

// This warp's map of tile t.  The last warp composes the CTA's and pushes it to every CTA of the cluster: 512 bytes a
// CTA, counted by the receiver's barrier.  The slot's last readers are past it: a CTA pushes tile t after it has
// received tile t - 1, hence after every CTA has pushed t - 1, which each does after reading tile t - 2.
__device__ __forceinline__ void publish(Shared &sh, const Map &own, int t, int S, uint32_t rank)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, slot = t % kSlots;
    if (w < kWarps - 1 || S == 1) {
        sh.warps[slot][w][lane] = own.packed();
        if (S > 1)   // two barriers in turn: a warp arrives for tile t + 1 once it has received tile t
            asm volatile("barrier.cta.arrive %0, %1;" ::"r"(1 + (t & 1)), "n"(kThreads) : "memory");
        return;
    }
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + (t & 1)), "n"(kThreads) : "memory");
    if (lane == 0)
        tc::bar_expect_tx(&sh.full[slot], S * 512);
    Map all;
#pragma unroll
    for (int i = 0; i < kWarps - 1; ++i)
        all.then(sh.warps[slot][i][lane]);
    all.then(own);
    for (int i = 0; i < S; ++i)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                         remote(&sh.ctas[slot][rank][lane], i)),
                     "f"(all.A.x), "f"(all.A.y), "f"(all.H.x), "f"(all.H.y), "r"(remote(&sh.full[slot], i))
                     : "memory");
}

// Waits for phase `parity` of a barrier that other CTAs' pushes complete.  Bounded: after about a second the CTA's
// abort word is set and later waits return at once; the results are then void.
__device__ __forceinline__ void wait_pushes(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    auto done = [&] {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}\n"
                     : "=r"(ok) : "r"(tc::smem_u32(bar)), "r"(parity), "r"(100000u) : "memory");
        return ok != 0;
    };
    if (done())
        return;
    const unsigned long long t0 = tc::global_ns();
    while (!done()) {
        if (*abort)
            return;
        if (tc::global_ns() - t0 > tc::kWaitNs) {
            *abort = 1;
            return;
        }
    }
}

// The state that enters this warp's rows of tile t; advances `carry` past the cluster's tiles.
__device__ __forceinline__ float2 receive(Shared &sh, float2 &carry, int t, int S, uint32_t rank)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, slot = t % kSlots;
    float2 in = carry;
    if (S == 1) {
        __syncthreads();   // every warp has published tile t
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i == w)
                in = carry;
            carry = Map(sh.warps[slot][i][lane])(carry);
        }
        return in;
    }
    wait_pushes(&sh.full[slot], t / kSlots & 1, &sh.abort);
    for (int i = 0; i < S; ++i) {
        if (i == (int)rank)
            in = carry;
        carry = Map(sh.ctas[slot][i][lane])(carry);
    }
    for (int i = 0; i < w; ++i)
        in = Map(sh.warps[slot][i][lane])(in);
    return in;
}

template <typename Tx, typename Tg, typename To, bool ALIGNED, int RPT, int STAGES>
__global__ void __launch_bounds__(kThreads, 2) scan_fwd_kernel(ScanArgs a, int tiles, int S)
{
    constexpr int R = kWarps * RPT;
    typedef Tile<Tx, R, ALIGNED> TX;
    typedef Tile<Tg, R, ALIGNED> TG;
    constexpr int kStage = TX::kBytes + TG::kBytes;
    extern __shared__ __align__(128) char smem[];
    __shared__ Shared sh;

    const int unit = blockIdx.x / S, n = unit / tiles, d0 = (unit - n * tiles) * kCols;
    const uint32_t rank = S > 1 ? cluster_rank() : 0;
    int64_t begin;
    int len;
    if (!sequence_rows(a, n, begin, len))
        return;                                       // the whole cluster leaves here
    const Pair<ALIGNED> pair(d0, a.D);
    const bool full = d0 + kCols <= a.D;
    const int w = threadIdx.x >> 5;
    const int64_t state = (int64_t)n * a.D;
    const Tx *x = static_cast<const Tx *>(a.x) + begin * a.ldx + d0;
    const Tg *g = static_cast<const Tg *>(a.g) + begin * a.ldg + d0;
    float2 carry = pair.state(a.h0, state);
    const int step = S * R, iters = (len + step - 1) / step;
    auto load = [&](int it) {
        if (it < iters) {
            char *st = smem + it % STAGES * kStage;
            const int r0 = it * step + rank * R;
            TX::template load<1>(st, x, a.ldx, r0, len, a.D - d0);
            TG::template load<1>(st + TX::kBytes, g, a.ldg, r0, len, a.D - d0);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
        load(i);
    if (S > 1)
        open_cluster(sh);
    for (int it = 0; it < iters; ++it) {
        copy_wait<STAGES - 2>();
        __syncthreads();                              // tile `it` is here, and nobody reads tile it - 1 any more
        load(it + STAGES - 1);
        const char *st = smem + it % STAGES * kStage;
        const int r0 = it * step + rank * R + w * RPT;
        Map row[RPT], own;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            row[i].A = decay2(TG::read(st + TX::kBytes, w * RPT + i, g, a.ldg, r0 + i));
            row[i].H = TX::read(st, w * RPT + i, x, a.ldx, r0 + i);
            own.then(row[i]);
        }
        publish(sh, own, it, S, rank);
        float2 s = receive(sh, carry, it, S, rank);
        To *h = static_cast<To *>(a.h) + (begin + r0) * a.D;
        const int left = len - r0;
        auto emit = [&](auto tag) {
            constexpr bool whole = decltype(tag)::value;
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                s = row[i](s);
                if (whole || i < left)
                    pair.template store<whole>(h + (int64_t)i * a.D, s);
            }
        };
        if (left >= RPT && full)
            emit(std::true_type());
        else
            emit(std::false_type());
    }
    if (a.ht && rank == 0 && w == 0)
        pair.put_state(a.ht, state, carry);
    if (S > 1)
        close_cluster(sh, a.status);
}

template <typename Tx, typename Tg, typename To, bool ALIGNED, int RPT, int STAGES>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(ScanArgs a, int tiles, int S)
{
    constexpr int R = kWarps * RPT;
    typedef Tile<Tg, R, ALIGNED> TG;
    typedef Tile<To, R, ALIGNED> TO;
    constexpr int kStage = TG::kBytes + 2 * TO::kBytes;
    extern __shared__ __align__(128) char smem[];
    __shared__ Shared sh;

    const int unit = blockIdx.x / S, n = unit / tiles, d0 = (unit - n * tiles) * kCols;
    const uint32_t rank = S > 1 ? cluster_rank() : 0;
    int64_t begin;
    int len;
    if (!sequence_rows(a, n, begin, len))
        return;
    const Pair<ALIGNED> pair(d0, a.D);
    const bool full = d0 + kCols <= a.D;
    const int w = threadIdx.x >> 5;
    const int64_t state = (int64_t)n * a.D;
    const Tg *g = static_cast<const Tg *>(a.g) + begin * a.ldg + d0;
    const To *h = static_cast<const To *>(a.h_in) + begin * a.D + d0;
    const To *dh = static_cast<const To *>(a.dh) + begin * a.D + d0;
    float2 carry = pair.state(a.dht, state);
    const float2 h0 = pair.state(a.h0, state);
    const int step = S * R, iters = (len + step - 1) / step;
    // position p of the walk is row len - 1 - p
    auto load = [&](int it) {
        if (it < iters) {
            char *st = smem + it % STAGES * kStage;
            const int last = len - 1 - (it * step + (int)rank * R);
            TG::template load<-1>(st, g, a.ldg, last, len, a.D - d0);
            TO::template load<-1>(st + TG::kBytes, dh, a.D, last, len, a.D - d0);
            TO::template load<-1>(st + TG::kBytes + TO::kBytes, h, a.D, last - 1, len, a.D - d0);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
        load(i);
    if (S > 1)
        open_cluster(sh);
    for (int it = 0; it < iters; ++it) {
        copy_wait<STAGES - 2>();
        __syncthreads();
        load(it + STAGES - 1);
        const char *st = smem + it % STAGES * kStage;
        const int last = len - 1 - (it * step + (int)rank * R + w * RPT);
        float2 dec[RPT], up[RPT];
        Map own;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            dec[i] = decay2(TG::read(st, w * RPT + i, g, a.ldg, last - i));
            up[i] = TO::read(st + TG::kBytes, w * RPT + i, dh, a.D, last - i);
            own.A = mul2(own.A, dec[i]);
            own.H = mul2(dec[i], add2(own.H, up[i]));
        }
        publish(sh, own, it, S, rank);
        float2 mu = receive(sh, carry, it, S, rank);
        Tx *dx = static_cast<Tx *>(a.dx) + (begin + last) * a.lddx;
        Tg *dg = static_cast<Tg *>(a.dg) + (begin + last) * a.lddg;
        auto emit = [&](auto tag) {
            constexpr bool whole = decltype(tag)::value;
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                float2 prev = TO::read(st + TG::kBytes + TO::kBytes, w * RPT + i, h, a.D, last - i - 1);
                if (!whole && i == last)
                    prev = h0;
                const float2 lam = add2(up[i], mu);
                mu = mul2(dec[i], lam);
                if (whole || i <= last) {
                    pair.template store<whole>(dx - (int64_t)i * a.lddx, lam);
                    pair.template store<whole>(dg - (int64_t)i * a.lddg, mul2(mu, prev));
                }
            }
        };
        if (last >= RPT && full)
            emit(std::true_type());
        else
            emit(std::false_type());
    }
    if (a.dh0 && rank == 0 && w == 0)
        pair.put_state(a.dh0, state, carry);
    if (S > 1)
        close_cluster(sh, a.status);
}

// CTAs of a cluster: as many as run at once (two CTAs an SM), up to one time slice of R rows each.  More would wait
// for a second wave, whose clusters start when the first have ended: 8 x 4096 rows of 2048 channels, backward, run in
// 115 us with 256 CTAs and in 152 us with 512.
int cluster_size(int64_t units, int64_t rows, int R)
{
    const int64_t fit = 2 * sm_count() / std::max<int64_t>(units, 1), slices = (rows + R - 1) / R;
    return (int)std::max<int64_t>(1, std::min<int64_t>({fit, slices, kMaxCluster}));
}

template <typename K>
cudaError_t launch(K kernel, const ScanArgs &a, int R, int smem, cudaStream_t s)
{
    const int tiles = (a.D + kCols - 1) / kCols;
    const int S = cluster_size((int64_t)a.N * tiles, a.T, R);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.N * tiles * S);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, tiles, S);
}

// Whether rows of `elem`-byte elements start and step in 16-byte units.
bool units16(int64_t ld, int D, int elem) { return ld * elem % 16 == 0 && (int64_t)D * elem % 16 == 0; }

template <typename Tx, typename Tg, typename To, bool ALIGNED>
cudaError_t fwd(const ScanArgs &a, cudaStream_t s)
{
    constexpr int RPT = sizeof(Tx) + sizeof(Tg) > 4 ? 8 : 16, R = kWarps * RPT, STAGES = 3;
    return launch(scan_fwd_kernel<Tx, Tg, To, ALIGNED, RPT, STAGES>, a, R,
                  STAGES * (Tile<Tx, R, ALIGNED>::kBytes + Tile<Tg, R, ALIGNED>::kBytes), s);
}

template <typename Tx, typename Tg, typename To, bool ALIGNED>
cudaError_t bwd(const ScanArgs &a, cudaStream_t s)
{
    constexpr int RPT = 8, R = kWarps * RPT, STAGES = 3;
    return launch(scan_bwd_kernel<Tx, Tg, To, ALIGNED, RPT, STAGES>, a, R,
                  STAGES * (Tile<Tg, R, ALIGNED>::kBytes + 2 * Tile<To, R, ALIGNED>::kBytes), s);
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs &a, int dtype, cudaStream_t s)
{
    return by_types(dtype, [&](auto x, auto g, auto o) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(g)> Tg;
        typedef std::remove_pointer_t<decltype(o)> To;
        const bool ok = units16(a.ldx, a.D, sizeof(Tx)) && units16(a.ldg, a.D, sizeof(Tg));
        return ok ? fwd<Tx, Tg, To, true>(a, s) : fwd<Tx, Tg, To, false>(a, s);
    });
}

cudaError_t launch_scan_bwd(const ScanArgs &a, int dtype, cudaStream_t s)
{
    return by_types(dtype, [&](auto x, auto g, auto o) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(g)> Tg;
        typedef std::remove_pointer_t<decltype(o)> To;
        const bool ok = units16(a.ldg, a.D, sizeof(Tg)) && units16(a.D, a.D, sizeof(To)) &&
                        units16(a.lddx, a.D, sizeof(Tx)) && units16(a.lddg, a.D, sizeof(Tg));
        return ok ? bwd<Tx, Tg, To, true>(a, s) : bwd<Tx, Tg, To, false>(a, s);
    });
}

}  // namespace gla
