// Vector-state gated linear recurrence, forward and backward, in one pass over the data.
//
// h_t = a_t h_{t-1} + x_t with a_t = exp(g_t) is a chain of affine maps, and maps compose: rows r..s together take
// the entering state h to A h + H, with A their total decay and H the state they reach from zero.  So the time axis is
// cut: a thread folds RPT consecutive rows of two channels into (A, H), the CTA composes its warps'
// maps, a cluster of S CTAs composes its CTAs' maps through distributed shared memory, and the state entering every
// thread's rows follows; the thread then runs its rows again from that state (decays kept in registers, inputs still
// in shared memory) and writes them.  The cluster walks the sequence S * R rows at a time and carries the state.
// The backward is the same chain from the last row to the first: mu_t = a_t (dh_t + mu_{t+1}).
//
// Every input is read once and every output written once.  The order of all sums is fixed by the shape (and the SMs).
//
// HBM bounds it where there is enough to do: 65536 rows of 4096 channels, 16 bits, 248-257 us (6.3-6.5 TB/s; a copy
// runs at 6.8), the backward of 65536 x 2048 205 us (6.5).  A tile of 128 rows by 64 channels costs a CTA 0.9 us alone
// and 2 us beside another on its SM (16.3 instructions an element, 24.6 in the backward), an exchange between CTAs 0.45;
// few channels of long sequences are bound by that chain (65536 x 512: 72 us), short ones by starting it.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "api_common.h"
#include "gla_internal.h"
#include "layer_internal.h"
#include "tc_ptx.cuh"

namespace gla {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kCols = 64;       // channels of a CTA: two per lane
constexpr int kMaxCluster = 12;   // 65536 rows of 512 channels: 4 CTAs 174 us, 8: 96, 12: 72, but 14: 129 and 16: 115
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

// How rows lie in memory: on whole 16-byte units; elsewhere, but with their channels in whole pairs; anywhere.
enum Rows { kUnits, kPairs, kAnywhere };

// One R x kCols tile of a row-strided tensor in shared memory: row j is row r0 + DIR j of the sequence.  Rows on whole
// 16-byte units lie as they are.  Others start anywhere in a unit and are copied by units, from the one that holds their
// first byte; their pitch in shared memory differs from the step in memory by a multiple of 16, so that every row
// starts as far into a unit as in memory and row j is found at a fixed step from row 0 (an address worked out for each
// row and copy was 17% more instructions; 16 bits, 2 x 8192 rows of 1539 channels: forward 50 -> 47 us,
// with twelve rows a thread the backward 86 -> 74).
template <typename T, int R, Rows ROWS, int DIR>
struct Tile {
    static constexpr int kElem = (int)sizeof(T), kWhole = kCols * kElem / 16;   // units of a row that starts on one
    static constexpr int kPitch = 16 * kWhole + (ROWS == kUnits ? 0 : 16);      // the least pitch
    static constexpr int kBytes = ROWS == kUnits ? R * kPitch : (R * (kPitch + 16 - kElem) + 31) / 16 * 16;
    const T *src;     // the sequence's first row at the tile's first channel
    int64_t ld;       // bytes between rows
    int pitch;

    __device__ __forceinline__ Tile(const T *src, int64_t stride)
        : src(src), ld(stride * kElem), pitch(ROWS == kUnits ? kPitch : kPitch + (int)(DIR * ld & 15)) {}
    // Bytes into a unit at which row r starts (only the low bits of its address count).
    __device__ __forceinline__ int shift(int r) const
    {
        return ROWS == kUnits ? 0 : (int)(((uint32_t)reinterpret_cast<uintptr_t>(src) + (uint32_t)r * (uint32_t)ld) & 15);
    }

    // Rows outside [0, len) are zeros; channels from `cols` on are anything.  A thread copies from one unit of the rows
    // kStep apart, which start equally far into a unit; the units past kWhole that shifted rows end in go one a thread.
    __device__ __forceinline__ void load(char *dst, int r0, int len, int cols) const
    {
        constexpr int kStep = kThreads / kWhole;
        static_assert(R % kStep == 0 && kStep * kElem % 16 == 0 && R <= kThreads);
        const char *base = reinterpret_cast<const char *>(src);
        const int lead = shift(r0), width = min(kCols, cols) * kElem;
        const bool all = (unsigned)r0 < (unsigned)len && (unsigned)(r0 + DIR * (R - 1)) < (unsigned)len;
        auto unit = [&](int j) { return dst + ((lead + j * pitch) & ~15); };   // row j's first
        auto bytes = [&](int sh, int u) { return max(0, min(16, sh + width - 16 * u)); };
        const int u = threadIdx.x % kWhole, j0 = threadIdx.x / kWhole, r = r0 + DIR * j0, sh = shift(r), n = bytes(sh, u);
        const char *p = base + r * ld - sh + 16 * u;
        const int64_t step = (int64_t)DIR * kStep * ld;
        char *q = unit(j0) + 16 * u;
        if (ROWS == kUnits && all && cols >= kCols) {
#pragma unroll
            for (int j = 0; j < R; j += kStep)
                copy16(q + j * pitch, p + j / kStep * step);
        } else if (ROWS != kUnits && all) {
            if (n > 0)
#pragma unroll
                for (int j = 0; j < R; j += kStep)
                    copy16(q + j * pitch, p + j / kStep * step, n);
        } else {
#pragma unroll
            for (int j = 0; j < R; j += kStep) {
                const bool ok = n > 0 && (unsigned)(r + DIR * j) < (unsigned)len;
                copy16(q + j * pitch, ok ? p : base - shift(0), ok ? n : 0);
                p += step;
            }
        }
        if (ROWS != kUnits && threadIdx.x < R) {
            const int j = threadIdx.x, r = r0 + DIR * j, sh = shift(r), n = bytes(sh, kWhole);
            const bool ok = n > 0 && (all || (unsigned)r < (unsigned)len);
            if (ok || !all)
                copy16(unit(j) + 16 * kWhole, ok ? base + r * ld - sh + 16 * kWhole : base - shift(0), ok ? n : 0);
        }
    }

    // Where the tile's rows from j on are, row j being row r of the sequence; then the lane's two channels of the row i
    // further on: 2 l and 2 l + 1, or l and l + 32 for rows anywhere.
    __device__ __forceinline__ const char *at(const char *tile, int j, int r) const
    {
        const int lane = threadIdx.x & 31;
        return tile + shift(r - DIR * j) + j * pitch + (ROWS == kAnywhere ? kElem : 2 * kElem) * lane;
    }
    __device__ __forceinline__ float2 read(const char *rows, int i) const
    {
        const char *row = rows + i * pitch;
        if constexpr (ROWS == kAnywhere) {
            const T *p = reinterpret_cast<const T *>(row);
            return make_float2(widen(p[0]), widen(p[32]));
        } else if constexpr (kElem == 4) {
            return *reinterpret_cast<const float2 *>(row);
        } else {
            return widen2<T>(*reinterpret_cast<const uint32_t *>(row));
        }
    }
};

// The lane's two channels, and the stores of a pair.
template <bool PAIRED>
struct Pair {
    int d[2];
    bool on[2];
    __device__ __forceinline__ Pair(int d0, int D)
    {
        const int lane = threadIdx.x & 31;
        d[0] = d0 + (PAIRED ? 2 * lane : lane);
        d[1] = d0 + (PAIRED ? 2 * lane + 1 : lane + 32);
        on[0] = d[0] < D;
        on[1] = d[1] < D;
    }
    template <bool WHOLE, typename T>   // WHOLE: both channels exist
    __device__ __forceinline__ void store(T *row, float2 v) const
    {
        if constexpr (PAIRED) {
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

__device__ __forceinline__ float2 exp2_fast2(float2 t) { return make_float2(exp2_fast(t.x), exp2_fast(t.y)); }
__device__ __forceinline__ float2 log2_decay(float2 g) { return mul2(g, make_float2(kLog2e, kLog2e)); }
__device__ __forceinline__ float2 decay2(float2 g) { return exp2_fast2(log2_decay(g)); }

// An affine map h -> a (a h) + H of a lane's two channels.  a is the root of the rows' total decay A, from the sum of
// their gates, and at most the largest fp32 value.  Gates may rise and fall by more than an exponential's range and
// still leave the states in theirs; then A may be no fp32 value (or, as a product of decays, come back from 0 or infinity
// as something else), but its root is one wherever a normal h leaves A h in range, and a (a h) is right in one rounding
// more.  An h of zero stays zero, whatever a is.  Against products of decays: the same time where HBM bounds it, 71.6 ->
// 72.3 us for 65536 x 512, and fp32 outputs nearer to fp64 (3.0e-7 -> 2.3e-7 relative), as a sum rounds less than a product.
struct Map {
    float2 a, H;
    __device__ __forceinline__ Map() : a{1.f, 1.f}, H{0.f, 0.f} {}
    __device__ __forceinline__ Map(float4 v) : a{v.x, v.y}, H{v.z, v.w} {}
    __device__ __forceinline__ float4 packed() const { return make_float4(a.x, a.y, H.x, H.y); }
    __device__ __forceinline__ void set_decay(float2 sum)   // of the rows' log2 decays
    {
        a = exp2_fast2(mul2(sum, make_float2(0.5f, 0.5f)));
        bound();
    }
    __device__ __forceinline__ void bound() { a = make_float2(fminf(a.x, FLT_MAX), fminf(a.y, FLT_MAX)); }
    __device__ __forceinline__ void then(const Map &m)   // this map, then m (bound() after the last)
    {
        a = mul2(a, m.a);
        H = m(H);
    }
    __device__ __forceinline__ float2 operator()(float2 h) const { return fma2(a, mul2(a, h), H); }
};

struct Shared {
    float4 warps[kSlots][kWarps][32];       // the maps of a tile's warps
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

// This warp's map of tile t.  The last warp composes the CTA's and pushes it to every CTA of the cluster (`ctas`, S
// rows a slot): 512 bytes a CTA, counted by the receiver's barrier.  The slot's last readers are past it: a CTA pushes
// tile t after it has received tile t - 1, hence after every CTA has pushed t - 1, which each does after reading tile
// t - 2.
__device__ __forceinline__ void publish(Shared &sh, float4 *ctas, const Map &own, int t, int S, uint32_t rank)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, slot = t % kSlots;
    if (w < kWarps - 1 || S == 1) {
        sh.warps[slot][w][lane] = own.packed();
        if (S > 1) {   // two barriers in turn: a warp arrives for tile t + 1 once it has received tile t
            if (t & 1)
                asm volatile("barrier.cta.arrive 1, %0;" ::"n"(kThreads) : "memory");
            else
                asm volatile("barrier.cta.arrive 2, %0;" ::"n"(kThreads) : "memory");
        }
        return;
    }
    if (t & 1)
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(kThreads) : "memory");
    else
        asm volatile("barrier.cta.sync 2, %0;" ::"n"(kThreads) : "memory");
    if (lane == 0)
        tc::bar_expect_tx(&sh.full[slot], S * 512);
    Map all;
#pragma unroll
    for (int i = 0; i < kWarps - 1; ++i)
        all.then(sh.warps[slot][i][lane]);
    all.then(own);
    all.bound();
    for (int i = 0; i < S; ++i)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                         remote(ctas + (slot * S + rank) * 32 + lane, i)),
                     "f"(all.a.x), "f"(all.a.y), "f"(all.H.x), "f"(all.H.y), "r"(remote(&sh.full[slot], i))
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
__device__ __forceinline__ float2 receive(Shared &sh, const float4 *ctas, float2 &carry, int t, int S, uint32_t rank)
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
        carry = Map(ctas[(slot * S + i) * 32 + lane])(carry);
    }
    for (int i = 0; i < w; ++i)
        in = Map(sh.warps[slot][i][lane])(in);
    return in;
}

// What a CTA does with its tiles.  Position p of the forward's walk is row p of the sequence.
template <typename Tx, typename Tg, typename To, Rows ROWS, int RPT_>
struct Forward {
    static constexpr int RPT = RPT_, R = kWarps * RPT;
    typedef Tile<Tx, R, ROWS, 1> TX;
    typedef Tile<Tg, R, ROWS, 1> TG;
    static constexpr int kStage = TX::kBytes + TG::kBytes;
    typedef Pair<ROWS != kAnywhere> Lane;
    float2 dec[RPT], in[RPT];
    const TX x;
    const TG g;
    To *h;
    int len;
    bool full;   // the tile's channels all exist

    __device__ __forceinline__ Forward(const ScanArgs &a, int64_t begin, int len, int d0, const Lane &, int64_t)
        : x(static_cast<const Tx *>(a.x) + begin * a.ldx + d0, a.ldx),
          g(static_cast<const Tg *>(a.g) + begin * a.ldg + d0, a.ldg), h(static_cast<To *>(a.h) + begin * a.D), len(len), full(d0 + kCols <= a.D) {}
    static __device__ __forceinline__ const float *start(const ScanArgs &a) { return a.h0; }
    static __device__ __forceinline__ float *end(const ScanArgs &a) { return a.ht; }
    __device__ __forceinline__ void load(const ScanArgs &a, char *st, int p, int d0) const
    {
        x.load(st, p, len, a.D - d0);
        g.load(st + TX::kBytes, p, len, a.D - d0);
    }
    // Positions p.. of the walk, rows j.. of the tile.
    __device__ __forceinline__ Map fold(const char *st, int p, int j)
    {
        const char *gs = g.at(st + TX::kBytes, j, p), *xs = x.at(st, j, p);
        Map own;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float2 t = log2_decay(g.read(gs, i));
            dec[i] = exp2_fast2(t);
            in[i] = x.read(xs, i);
            sum = add2(sum, t);
            own.H = fma2(dec[i], own.H, in[i]);
        }
        own.set_decay(sum);
        return own;
    }
    template <bool WHOLE>
    __device__ __forceinline__ void put(const ScanArgs &a, float2 s, int p, const Lane &lane) const
    {
        To *at = h + (int64_t)p * a.D;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            s = fma2(dec[i], s, in[i]);
            if (WHOLE || p + i < len)
                lane.template store<WHOLE>(at + (int64_t)i * a.D, s);
        }
    }
    __device__ __forceinline__ void emit(const ScanArgs &a, const char *, float2 s, int p, int, const Lane &lane) const
    {
        if (full && p + RPT <= len)
            put<true>(a, s, p, lane);
        else
            put<false>(a, s, p, lane);
    }
};

// Position p of the backward's walk is row len - 1 - p; its state is mu.
template <typename Tx, typename Tg, typename To, Rows ROWS, int RPT_>
struct Backward {
    static constexpr int RPT = RPT_, R = kWarps * RPT;
    typedef Tile<Tg, R, ROWS, -1> TG;
    typedef Tile<To, R, ROWS, -1> TO;
    static constexpr int kStage = TG::kBytes + 2 * TO::kBytes;
    typedef Pair<ROWS != kAnywhere> Lane;
    float2 dec[RPT], up[RPT];
    const TG g;
    const TO h, dh;
    Tx *dx;
    Tg *dg;
    int len;
    bool full;
    const float2 h0;

    __device__ __forceinline__ Backward(const ScanArgs &a, int64_t begin, int len, int d0, const Lane &lane, int64_t state)
        : g(static_cast<const Tg *>(a.g) + begin * a.ldg + d0, a.ldg),
          h(static_cast<const To *>(a.h_in) + begin * a.D + d0, a.D),
          dh(static_cast<const To *>(a.dh) + begin * a.D + d0, a.D), dx(static_cast<Tx *>(a.dx) + begin * a.lddx),
          dg(static_cast<Tg *>(a.dg) + begin * a.lddg), len(len), full(d0 + kCols <= a.D), h0(lane.state(a.h0, state)) {}
    static __device__ __forceinline__ const float *start(const ScanArgs &a) { return a.dht; }
    static __device__ __forceinline__ float *end(const ScanArgs &a) { return a.dh0; }
    __device__ __forceinline__ void load(const ScanArgs &a, char *st, int p, int d0) const
    {
        const int r = len - 1 - p;
        g.load(st, r, len, a.D - d0);
        dh.load(st + TG::kBytes, r, len, a.D - d0);
        h.load(st + TG::kBytes + TO::kBytes, r - 1, len, a.D - d0);
    }
    __device__ __forceinline__ Map fold(const char *st, int p, int j)
    {
        const int r = len - 1 - p;
        const char *gs = g.at(st, j, r), *ds = dh.at(st + TG::kBytes, j, r);
        Map own;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float2 t = log2_decay(g.read(gs, i));
            dec[i] = exp2_fast2(t);
            up[i] = dh.read(ds, i);
            sum = add2(sum, t);
            own.H = mul2(dec[i], add2(own.H, up[i]));
        }
        own.set_decay(sum);
        return own;
    }
    template <bool WHOLE>
    __device__ __forceinline__ void put(const ScanArgs &a, const char *st, float2 mu, int r, int j, const Lane &lane) const
    {
        Tx *to_x = dx + (int64_t)r * a.lddx;
        Tg *to_g = dg + (int64_t)r * a.lddg;
        const char *hs = h.at(st + TG::kBytes + TO::kBytes, j, r - 1);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            float2 prev = h.read(hs, i);
            if (!WHOLE && i == r)
                prev = h0;
            const float2 lam = add2(up[i], mu);
            mu = mul2(dec[i], lam);
            if (WHOLE || i <= r) {
                lane.template store<WHOLE>(to_x - (int64_t)i * a.lddx, lam);
                lane.template store<WHOLE>(to_g - (int64_t)i * a.lddg, mul2(mu, prev));
            }
        }
    }
    __device__ __forceinline__ void emit(const ScanArgs &a, const char *st, float2 mu, int p, int j, const Lane &lane) const
    {
        const int r = len - 1 - p;
        if (full && r >= RPT)
            put<true>(a, st, mu, r, j, lane);
        else
            put<false>(a, st, mu, r, j, lane);
    }
};

// Tiles in shared memory at a time: three where two CTAs of an SM have room for them (16-bit forward), else two.
template <typename Role>
constexpr int kStages = Role::kStage <= 32768 ? 3 : 2;

template <typename Role>
__global__ void __launch_bounds__(kThreads, 2) scan_tiles(ScanArgs a, int tiles, int S)
{
    constexpr int RPT = Role::RPT, R = Role::R, STAGES = kStages<Role>;
    extern __shared__ __align__(128) char smem[];     // STAGES tiles, then the cluster's maps
    __shared__ Shared sh;
    float4 *ctas = reinterpret_cast<float4 *>(smem + STAGES * Role::kStage);

    const int unit = blockIdx.x / S, n = unit / tiles, d0 = (unit - n * tiles) * kCols;
    const uint32_t rank = S > 1 ? cluster_rank() : 0;
    if (S > 1)
        open_cluster(sh);
    tc::grid_dep_wait();   // launched early (0.1 to 0.4 us less): nothing above reads or writes global memory
    int64_t begin;
    int len;
    if (!sequence_rows(a, n, begin, len) || len <= a.alone)
        return;                                       // the whole cluster leaves here
    const typename Role::Lane lane(d0, a.D);
    const int w = threadIdx.x >> 5;
    const int64_t state = (int64_t)n * a.D;
    Role role(a, begin, len, d0, lane, state);
    float2 carry = lane.state(Role::start(a), state);
    const int step = S * R, iters = (len + step - 1) / step;
    auto load = [&](int t) {
        if (t < iters)
            role.load(a, smem + t % STAGES * Role::kStage, t * step + rank * R, d0);
        copy_commit();
    };
#pragma unroll
    for (int t = 0; t < STAGES - 1; ++t)
        load(t);
    for (int t = 0; t < iters; ++t) {
        copy_wait<STAGES - 2>();
        __syncthreads();                              // tile t is here, and nobody reads tile t - 1 any more
        load(t + STAGES - 1);
        const char *st = smem + t % STAGES * Role::kStage;
        const int p = t * step + rank * R + w * RPT;
        publish(sh, ctas, role.fold(st, p, w * RPT), t, S, rank);
        role.emit(a, st, receive(sh, ctas, carry, t, S, rank), p, w * RPT, lane);
    }
    if (Role::end(a) && rank == 0 && w == 0)
        lane.put_state(Role::end(a), state, carry);
    if (S > 1)
        close_cluster(sh, a.status);
}

// The lane's two channels of a row as they lie in memory: 2 l and 2 l + 1 in one load where rows start and step in
// whole pairs (PAIRED), else l and l + 32 one by one.
template <typename T, bool PAIRED>
struct Two {
    typedef std::conditional_t<PAIRED, std::conditional_t<sizeof(T) == 4, float2, uint32_t>, T> Raw;
    Raw v[PAIRED ? 1 : 2];

    __device__ __forceinline__ void load(const T *p, bool on0, bool on1)   // p: the lane's first channel
    {
        if constexpr (PAIRED) {
            v[0] = on0 ? *reinterpret_cast<const Raw *>(p) : Raw{};
        } else {
            v[0] = on0 ? p[0] : T(0.f);
            v[1] = on1 ? p[32] : T(0.f);
        }
    }
    __device__ __forceinline__ float2 get() const
    {
        if constexpr (!PAIRED)
            return make_float2(widen(v[0]), widen(v[1]));
        else if constexpr (sizeof(T) == 4)
            return v[0];
        else
            return widen2<T>(v[0]);
    }
    static __device__ __forceinline__ void store(T *p, float2 f, bool on0, bool on1)
    {
        if constexpr (PAIRED) {
            if (on0) {
                if constexpr (sizeof(T) == 4)
                    *reinterpret_cast<float2 *>(p) = f;
                else
                    *reinterpret_cast<uint32_t *>(p) = narrow2<T>(f);
            }
        } else {
            if (on0)
                p[0] = narrow<T>(f.x);
            if (on1)
                p[32] = narrow<T>(f.y);
        }
    }
};


// Few rows, or so many channels that they alone fill the GPU: a thread walks two channels of a sequence, kAhead rows
// at a time, whose loads are under way together (512 x 64 rows of 2048 channels, 16 bits: 64 us, 6.3 TB/s).
constexpr int kAhead = 8;

template <typename Tx, typename Tg, typename To, bool PAIRED>
__global__ void __launch_bounds__(128) scan_fwd_rows(ScanArgs a, int tiles)
{
    tc::grid_dep_wait();
    const int n = blockIdx.x / tiles, c = (blockIdx.x % tiles) * 4 + (threadIdx.x >> 5), d0 = c * kCols;
    int64_t begin;
    int len;
    if (!sequence_rows(a, n, begin, len) || len > a.alone || d0 >= a.D)
        return;
    const Pair<PAIRED> lane(d0, a.D);
    const int64_t state = (int64_t)n * a.D;
    const Tx *x = static_cast<const Tx *>(a.x) + begin * a.ldx + lane.d[0];
    const Tg *g = static_cast<const Tg *>(a.g) + begin * a.ldg + lane.d[0];
    To *h = static_cast<To *>(a.h) + begin * a.D + lane.d[0];
    float2 s = lane.state(a.h0, state);
    for (int r = 0; r < len; r += kAhead) {
        Two<Tx, PAIRED> xs[kAhead];
        Two<Tg, PAIRED> gs[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const bool ok = r + i < len;
            xs[i].load(x + (int64_t)i * a.ldx, ok && lane.on[0], ok && lane.on[1]);
            gs[i].load(g + (int64_t)i * a.ldg, ok && lane.on[0], ok && lane.on[1]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (r + i < len) {
                s = fma2(decay2(gs[i].get()), s, xs[i].get());
                Two<To, PAIRED>::store(h + (int64_t)i * a.D, s, lane.on[0], lane.on[1]);
            }
        x += kAhead * a.ldx;
        g += kAhead * a.ldg;
        h += kAhead * (int64_t)a.D;
    }
    if (a.ht)
        lane.put_state(a.ht, state, s);
}

template <typename Tx, typename Tg, typename To, bool PAIRED>
__global__ void __launch_bounds__(128) scan_bwd_rows(ScanArgs a, int tiles)
{
    tc::grid_dep_wait();
    const int n = blockIdx.x / tiles, c = (blockIdx.x % tiles) * 4 + (threadIdx.x >> 5), d0 = c * kCols;
    int64_t begin;
    int len;
    if (!sequence_rows(a, n, begin, len) || len > a.alone || d0 >= a.D)
        return;
    const Pair<PAIRED> lane(d0, a.D);
    const int64_t state = (int64_t)n * a.D;
    const float2 h0 = lane.state(a.h0, state);
    float2 mu = lane.state(a.dht, state);
    for (int r = len - 1; r >= 0; r -= kAhead) {
        const int64_t at = begin + r;
        const Tg *g = static_cast<const Tg *>(a.g) + at * a.ldg + lane.d[0];
        const To *dh = static_cast<const To *>(a.dh) + at * a.D + lane.d[0];
        const To *h = static_cast<const To *>(a.h_in) + (at - 1) * a.D + lane.d[0];
        Two<Tg, PAIRED> gs[kAhead];
        Two<To, PAIRED> ds[kAhead], hs[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            gs[i].load(g - (int64_t)i * a.ldg, i <= r && lane.on[0], i <= r && lane.on[1]);
            ds[i].load(dh - (int64_t)i * a.D, i <= r && lane.on[0], i <= r && lane.on[1]);
            hs[i].load(h - (int64_t)i * a.D, i < r && lane.on[0], i < r && lane.on[1]);
        }
        Tx *dx = static_cast<Tx *>(a.dx) + at * a.lddx + lane.d[0];
        Tg *dg = static_cast<Tg *>(a.dg) + at * a.lddg + lane.d[0];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i <= r) {
                const float2 lam = add2(ds[i].get(), mu);
                mu = mul2(decay2(gs[i].get()), lam);
                Two<Tx, PAIRED>::store(dx - (int64_t)i * a.lddx, lam, lane.on[0], lane.on[1]);
                Two<Tg, PAIRED>::store(dg - (int64_t)i * a.lddg, mul2(mu, i == r ? h0 : hs[i].get()), lane.on[0], lane.on[1]);
            }
    }
    if (a.dh0)
        lane.put_state(a.dh0, state, mu);
}

// Clusters of S = 1..kMaxCluster CTAs of a kernel that the current device runs at once.
struct Fit {
    std::mutex mu;
    std::atomic<bool> known[128] = {};
    int clusters[128][kMaxCluster + 1] = {};
};

// CTAs of a cluster, for `units` (sequence, channel tile) pairs of `rows` rows (a pack's mean): as many as run at once,
// up to one time slice of R rows each.  Where not even two each do, the clusters come in waves, and the shorter their
// walks, the less the last wave costs; on the other side are a start of about 1.5 tiles' time and an exchange of about
// 0.03 for each further CTA.  A last wave costs at least 0.6 of a full one (CTAs that share an SM no longer still wait
// for their own tiles).  The lengths of a pack differ, which leaves about half a walk at the end.  Measured for 1, 2
// and 4 CTAs, in us: 256 units of 4096 rows 70, 68, 69 (backward 116, 110, 111); 160 of 4096: 51, 58, 50; 1024 of 1024:
// 62, 76, 97; 512 of a pack of 128 to 8192 rows: 197, 182, 184 (at 8 rows a thread; 177 at 16).
int cluster_size(const int *fit, int64_t units, int64_t rows, int R, bool pack)
{
    int S = 1;
    for (int c = 2; c <= kMaxCluster && (c - 1) * R < rows; ++c)
        if (fit[c] >= units)
            S = c;
    if (S > 1)
        return S;
    double best = 0;
    for (int c : {1, 2, 4}) {
        if (fit[c] <= 0 || (c > 1 && (c - 1) * R >= rows))
            continue;
        const double walk = (double)((rows + c * R - 1) / (c * R)) * (1 + 0.03 * (c - 1)) + 1.5;
        const double full = (double)units / fit[c], whole = std::floor(full), part = full - whole;
        const double waves = pack ? full + 0.5 : full <= 1 ? 1 : whole + (part > 0 ? std::max(part, 0.6) : 0);
        if (c == 1 || waves * walk < best) {
            best = waves * walk;
            S = c;
        }
    }
    return S;
}

template <typename Role>
cudaError_t launch_tiles(const ScanArgs &a, cudaStream_t s)
{
    static Fit fit;
    constexpr int STAGES = kStages<Role>;
    auto kernel = scan_tiles<Role>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev >= 128)
        return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    auto shape = [&](int64_t units, int S) {
        at[0].val.clusterDim.x = S;
        cfg.gridDim = dim3((unsigned)(units * S));
        cfg.dynamicSmemBytes = STAGES * Role::kStage + (S > 1 ? kSlots * S * 512 : 0);
    };
    if (!fit.known[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(fit.mu);
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      STAGES * Role::kStage + kSlots * kMaxCluster * 512)) != cudaSuccess)
            return e;
        for (int S = 1; S <= kMaxCluster; ++S) {
            shape(1, S);
            int n = 0;
            fit.clusters[dev][S] = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
        }
        cudaGetLastError();
        fit.known[dev].store(true, std::memory_order_release);
    }
    const int tiles = (a.D + kCols - 1) / kCols;
    const int64_t units = (int64_t)a.N * tiles;
    const int S = cluster_size(fit.clusters[dev], units, a.cu ? a.T / a.N : a.T, Role::R, a.cu != nullptr);
    shape(units, S);
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, tiles, S);
}

// How rows that start `ld` elements of `elem` bytes apart, D of them channels, lie in memory.
Rows rows_of(int64_t ld, int D, int elem)
{
    return ld * elem % 16 == 0 && (int64_t)D * elem % 16 == 0 ? kUnits : ld % 2 == 0 && D % 2 == 0 ? kPairs : kAnywhere;
}

template <typename Tx, typename Tg, typename To, Rows ROWS>
cudaError_t fwd_tiles(const ScanArgs &a, cudaStream_t s)
{
    // Rows of a thread: the more the fewer exchanges, as registers and shared memory allow for two CTAs an SM; better
    // than a third tile under way (fp32, 5 x 41830 rows of 128 channels: 8 rows 93 us, 12 rows 75).
    constexpr int kBytes = sizeof(Tx) + sizeof(Tg);
    return launch_tiles<Forward<Tx, Tg, To, ROWS, ROWS == kUnits ? (kBytes == 8 ? 12 : 16)
                                                                 : kBytes == 4 ? 16 : kBytes == 6 ? 12 : 10>>(a, s);
}

template <typename Tx, typename Tg, typename To, Rows ROWS>
cudaError_t bwd_tiles(const ScanArgs &a, cudaStream_t s)
{
    constexpr int kBytes = sizeof(Tg) + 2 * sizeof(To);
    return launch_tiles<Backward<Tx, Tg, To, ROWS, ROWS == kUnits ? (kBytes == 6 ? 16 : 8)   // likewise
                                                                  : kBytes == 6 ? 12 : kBytes == 10 ? 8 : 6>>(a, s);
}

}  // namespace

// How a call's sequences are shared out: those of at most `rows` rows to threads that walk alone, the others to the
// tiles.  Alone is better for 16 rows at most (512 x 16 rows of 2048 channels: 19 us against 130), and for up to 128
// where there are enough channels to fill the GPU (256 x 128 rows of 2048 channels: 69 us against 83; 64 x 128 rows of
// 1024: 20 against 15).  The lengths of a pack are not known here: one of many sequences takes both kernels, each
// leaving the other's sequences alone; a pack of fewer takes the tiles, which split a long sequence too.
ScanShare scan_share(const ScanArgs &a)
{
    const int64_t channels = (int64_t)a.N * a.D;
    if (a.cu)
        return channels >= 8 * kCols * (int64_t)sm_count() ? ScanShare{64, true} : ScanShare{-1, true};
    const bool alone = a.T <= 16 || (a.T <= 128 && channels >= 2048 * (int64_t)a.T);
    return alone ? ScanShare{a.T, false} : ScanShare{-1, true};
}

cudaError_t launch_scan_fwd(const ScanArgs &a, int dtype, bool alone, cudaStream_t s)
{
    return by_types(dtype, [&](auto x, auto g, auto o) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(g)> Tg;
        typedef std::remove_pointer_t<decltype(o)> To;
        const Rows rows = std::max(rows_of(a.ldx, a.D, sizeof(Tx)), rows_of(a.ldg, a.D, sizeof(Tg)));
        if (alone) {
            const int tiles = (a.D + 4 * kCols - 1) / (4 * kCols);
            return rows != kAnywhere ? launch_early(scan_fwd_rows<Tx, Tg, To, true>, a.N * tiles, 128, s, a, tiles)
                                     : launch_early(scan_fwd_rows<Tx, Tg, To, false>, a.N * tiles, 128, s, a, tiles);
        }
        return rows == kUnits ? fwd_tiles<Tx, Tg, To, kUnits>(a, s)
               : rows == kPairs ? fwd_tiles<Tx, Tg, To, kPairs>(a, s) : fwd_tiles<Tx, Tg, To, kAnywhere>(a, s);
    });
}

cudaError_t launch_scan_bwd(const ScanArgs &a, int dtype, bool alone, cudaStream_t s)
{
    return by_types(dtype, [&](auto x, auto g, auto o) {
        typedef std::remove_pointer_t<decltype(x)> Tx;
        typedef std::remove_pointer_t<decltype(g)> Tg;
        typedef std::remove_pointer_t<decltype(o)> To;
        const Rows rows = std::max({rows_of(a.ldg, a.D, sizeof(Tg)), rows_of(a.D, a.D, sizeof(To)),
                                    rows_of(a.lddx, a.D, sizeof(Tx)), rows_of(a.lddg, a.D, sizeof(Tg))});
        if (alone) {
            const int tiles = (a.D + 4 * kCols - 1) / (4 * kCols);
            return rows != kAnywhere ? launch_early(scan_bwd_rows<Tx, Tg, To, true>, a.N * tiles, 128, s, a, tiles)
                                     : launch_early(scan_bwd_rows<Tx, Tg, To, false>, a.N * tiles, 128, s, a, tiles);
        }
        return rows == kUnits ? bwd_tiles<Tx, Tg, To, kUnits>(a, s)
               : rows == kPairs ? bwd_tiles<Tx, Tg, To, kPairs>(a, s) : bwd_tiles<Tx, Tg, To, kAnywhere>(a, s);
    });
}

}  // namespace gla
