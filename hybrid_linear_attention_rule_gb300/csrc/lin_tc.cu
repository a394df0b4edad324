// lin_tc.cu -- linear attention's jobs (lin.cuh) on the tensor cores: BF16 inputs, chunks of 64 tokens.
//
// Widths are padded to 128 by the copies' zero fill.  Everything is kept turned, channels of z in the 128 rows of an accumulator:
//     PT  = Y X^T                      scores, token j a row
//     ACC = Z^T [Yw | P]               the chunk's part of S^T [b, a] and of out^T [b, i], in one product of N = 192
//     O1  = S^T X^T                    what the state gives, S^T as an operand in tensor memory
// so that z, x and y are operands just as the copies laid them down, S^T lives in the registers of 512 threads (a row a lane, four
// threads a row) in FP32, and only the decayed scores P and keys Yw pass through shared memory, each as a sum of two or three BF16 numbers:
// the inputs are exact, so a product of three parts is FP32's accuracy, of two 2^-17.
//
// Roles of a CTA, joined by mbarriers: a copy warp (TMA), an MMA warp for ACC and one for PT and O1, so that no chain waits for the
// other's operands, eight warps that prepare P and Yw, sixteen that hold S, write its operand, fold ACC into it and put out rows.
// Each of them runs through its code once a chunk, so the code has to stay short: past some 60 KB of it the warps waited for instructions.
//
// The chunks of all (sequence, head) pairs stand in one line.  `plan_kernel` writes a record for each, where it lies and what its decays
// give, which the copies bring along.  The line is cut evenly over the CTAs ("pieces").  A piece that begins within a pair
// needs the state there: a first pass (STATES) runs the pieces that end within a pair for their state alone, `join_kernel` chains
// those of a pair, and the second pass starts from them.  The decay of a piece is one number a head, so the chain is a sum.
//
// What bounds it is neither HBM nor a pipe but the chain through a chunk: 8 k tokens of 32 heads take 135 us, 44 of them the first pass and 82 the
// second, 5,800 cycles a chunk with the tensor pipe busy for 1,800 and half of the issue slots used (HBM 39 %); 32 k tokens 470 us, 16 prompts of
// 32.6 k tokens 406.  With three parts (dq and dv, 8 k tokens) 300 us, 10,500 cycles a chunk, 2,200 of them products.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "lin.cuh"
#include "tc_ptx.cuh"

namespace k3kda {
namespace lin {
namespace {

using namespace tc;

constexpr int C = 64, D = 128, CTL = 128, PREP = 256, HOLD = 512, THREADS = CTL + PREP + HOLD;
constexpr int PREP_WARP = CTL / 32, HOLD_WARP = (CTL + PREP) / 32;
// A CTA's registers at its launch are THREADS x 72; the roles' shares may not be more.
constexpr int REG_CTL = 40, REG_PREP = 72, REG_HOLD = 80;
static_assert(CTL * REG_CTL + PREP * REG_PREP + HOLD * REG_HOLD <= THREADS * 72, "shares of the registers");
constexpr int COLS = 32, TOKENS = 16;                              // of the state and of the outputs that one of the holding threads has
constexpr uint32_t kTries = 1u << 20;            // a second or two
constexpr int MOST_PIECES = 160, WHOLE = 8;        // WHOLE: pairs of fewer chunks on average stay whole, where there are no more of them than CTAs

// How many pieces a line of U chunks of `pairs` pairs is worth, where up to `pieces` run at once: a CTA for each pair, or pieces of 16 chunks; where
// that leaves most SMs idle and pairs are long enough for a first pass, short ones of 2, or of 4 where pairs are long (their join walks over the
// pieces).  (One sequence, prefill and gradients in us, with pieces of 16, 4 and 2 chunks: 8 heads, 300 tokens 24 74, 36 87, 29 72; 600 tokens 38 116,
// 36 94, 30 78; 1,024 tokens 58 159, 36 94, 32 79; 2,048 tokens 81 194, 40 96, 38 103; 4,096 tokens 82 201, 47 132, 49 133; 2 heads of 8,192 tokens
// 84 192, 55 104, 72 144.  8 sequences of 512 tokens and 8 heads, whole 39 103, in pieces of 4 chunks 38 120.)
__device__ __forceinline__ long long worth(long long U, long long pairs, int pieces) {
    const long long fine = U / (U < 32 * pairs ? 2 : 4);
    return U >= WHOLE * pairs && min((long long)pieces, fine) >= 2 * pairs ? fine : max(pairs, U / 16);
}

enum Kind { kStates, kPlain, kFull };      // states alone; jobs whose operands are in two parts and that put out nothing but BF16 rows; any, in three parts

constexpr uint32_t TILE = C * 128;                                 // 64 rows of 64 BF16 values
// Shared memory: a ring of copies (y0 [x0] y1 [x1] z0 z1 [r0 r1]), parts of [Yw0 | Yw1 | P] (twice for the states, whose products then have no
// gap).  The rows put out stand in the place of x, once it has been used, until their copy has taken them.
template <Kind K> struct Map {
    static constexpr bool X = K != kStates;
    static constexpr int STAGES = K == kFull ? 2 : 3, SETS = K == kStates ? 2 : 1;
    static constexpr uint32_t Y = 0, XT = TILE, ATOM = (X ? 2 : 1) * TILE, Z = 2 * ATOM, R = Z + 2 * TILE, STAGE = R + (K == kFull ? 2 : 0) * TILE;
    static constexpr uint32_t OPS = STAGES * STAGE, PART = (X ? 3 : 2) * TILE, SET = K == kPlain ? 2 * PART + 2 * TILE : 3 * PART;
    static constexpr uint32_t INFO = OPS + SETS * SET;
};

// What a chunk's copies bring beside its rows; one of a direction and scale.  Its arrays are read in 16-byte pieces.
struct alignas(16) Record {
    float2 g[C];               // sums of the decays, as two floats; negative backward in time, so that d = g_i - g_j either way
    float c[C], w[C];
    float fi[C], fj[C];        // D_ij = fi[i] fj[j], the scale in fj, where the chunk's decay leaves both in range (`plain`)
    unsigned long long lost;   // tokens whose decay is NaN
    long long units;           // the chunk's decay,
    float keep;                // and its exponential
    int plain;
    int n, h, hk, t0, valid;   // hk: h / group
    int chunk, pos, chunks;    // of the pair's chunks: which in time, which in the line, how many
};
static_assert(sizeof(Record) % 16 == 0, "copied in 16-byte pieces");

struct Shared {
    Record rec[3];
    alignas(16) float own[3][C];       // P's diagonal, where it is kept apart
    unsigned char poison[3][D];        // of a z that is not finite: the channel's first such token in the job's direction, or NONE
    int dirty[3];              // whether there is one
    int dead;
    unsigned long long full[3], empty[3], pt_full, pt_free, prep_full, acc_full[2], acc_free[2], sop_full, o1_full, out_full, drain[2];
    uint32_t tmem;
};
constexpr int NONE = 255;
template <Kind K> constexpr uint32_t kSmem = Map<K>::INFO + sizeof(Shared) + 1024;
static_assert(kSmem<kStates> <= 232448 && kSmem<kPlain> <= 232448 && kSmem<kFull> <= 232448, "shared memory");

// tensor memory
constexpr uint32_t PT = 0, ACC = 64, ACC_O = ACC + D, O1 = 256, SOP = 320, ACC_STEP = 192;     // (states: two sets of ACC)

struct Head {                  // of a piece's state
    float keep;
    int ends_within, goes_on;  // whether the piece ends within a pair; whether it began within the same
};

struct TcArgs {
    CUtensorMap map[4];
    Call c;
    CUtensorMap out[3];        // the jobs' outputs, where they are BF16
    int x[3], y[3], z[3], r[3];        // the jobs' maps
    int rows;                  // of a copy's box
    int pieces;                // a job
    int fine;                  // those that the states were taken for: as many, or twice as many
    bool nested;               // pieces come in halves for another launch
    int of[3];                 // whose states a job begins its pieces with,
    bool turned[3];            // the other way round: its a is their b
    const Record *rec[3];      // the jobs'
    const long long *total;    // records of one
    Head *head;                // [jobs][fine]
    float *state;              // [jobs][fine][a][D]
    float *kept;               // likewise (one job), or null: the first states of the pairs that a piece leaves open, when they may be written over
};

template <int N> __device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// An arrival that waits for none of the thread's stores.  For barriers that hand over tensor memory alone: what the thread did there has
// ended (tcgen05.wait) and is fenced (tcgen05.fence) before; a releasing arrival would also wait until the rows stored last are in L2, which
// took 2 to 4 thousand cycles of a chunk.
__device__ __forceinline__ void arrive_relaxed(const unsigned long long &bar) {
    asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&bar)) : "memory");
}
// Stores under a predicate, without a branch around each.
__device__ __forceinline__ void store_if(bool on, char *to, __nv_bfloat16 v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.b16 [%0], %1;\n\t}" ::"l"(to), "h"(__bfloat16_as_ushort(v)), "r"((int)on) : "memory");
}
__device__ __forceinline__ void store_if(bool on, char *to, float v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.f32 [%0], %1;\n\t}" ::"l"(to), "f"(v), "r"((int)on) : "memory");
}
__device__ __forceinline__ uint32_t uniform(uint32_t x);
__device__ __forceinline__ char *uniform(const char *p) {
    const unsigned long long a = reinterpret_cast<unsigned long long>(p);
    return reinterpret_cast<char *>((unsigned long long)uniform((uint32_t)(a >> 32)) << 32 | uniform((uint32_t)a));
}
// A pair as BF16 numbers that add up to it; the rests are exact in FP32.
__device__ __forceinline__ uint32_t peel(float &x, float &y) {
    const uint32_t w = pack(x, y);
    x -= low(w);
    y -= high(w);
    return w;
}

__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// The same value in all lanes, and known to be: the MMA warps' addresses stay in uniform registers, whose instructions take nothing else.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// The smaller of a byte and `value` in its place, for many threads at once.
__device__ __forceinline__ void note_first(unsigned char *bytes, int at, unsigned value) {
    unsigned *const word = reinterpret_cast<unsigned *>(bytes + (at & ~3));
    const int shift = 8 * (at & 3);
    unsigned was = *word, now;
    do {
        now = was;
        if ((now >> shift & 255u) <= value) return;
        was = atomicCAS(word, now, (now & ~(255u << shift)) | value << shift);
    } while (was != now);
}

// A bounded wait of a whole warp, with the same answer for all its lanes; one that gives up ends the others' too.  (Short: the kernel's
// loops have to stay in the instruction cache.)
struct Waiter {
    volatile int *dead;
    __device__ __forceinline__ bool operator()(const unsigned long long &bar, int parity) const {
        const uint32_t at = smem_u32(&bar), odd = parity & 1;
        uint32_t i = kTries;
#pragma unroll 1
        while (!__all_sync(0xffffffffu, mbar_try_wait(at, odd)))
            if (__any_sync(0xffffffffu, --i == 0 || *dead)) {
                *dead = 1;
                return false;
            }
        return true;
    }
};

// The line of chunks: sequence n has max(1, ceil(len / C)) for each head, so that an empty one hands its state on.  Its bounds never
// run backwards, whatever the array holds (an end is at least the ends before it), so that no token is taken twice.
struct Line {
    const int32_t *cu;
    int T;
    __device__ __forceinline__ int bound(int i) const { return min(max(cu[i], 0), T); }
    __device__ __forceinline__ int length(int n, int &floor, int &begin) const {         // of sequence n; floor: the ends before it
        if (!cu) {
            begin = 0;
            return T;
        }
        begin = max(bound(n), floor);
        floor = max(floor, bound(n + 1));
        return floor - begin;
    }
};

// A call's kernels follow one another as programmatic dependents: the next one's CTAs may be set up while the one before still runs, and
// wait for its end before they read what it wrote.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct PlanArgs {
    const float *g;
    const int32_t *cu;
    int fixed, N, T, H, group, variants, reverse[2];
    float sp[2], sc[2], sw[2];
    Record *rec[2];
    long long *total;
};
constexpr int PLAN_THREADS = 256;

// The records: a warp a chunk, a CTA an even share of the line.  Latency bounds it: 7 us for 4,096 chunks, 10 with both directions.
__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const __grid_constant__ PlanArgs A) {
    __shared__ long long part[PLAN_THREADS / 32];
    __shared__ int part_end[PLAN_THREADS / 32], found[4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, N = A.N, H = A.H;
    let_next_start();
    const int per = (N + PLAN_THREADS - 1) / PLAN_THREADS, n0 = min(N, tid * per), n1 = min(N, n0 + per);
    const Line line{A.cu, A.T};
    int own_end = 0;
    if (A.cu)
        for (int n = n0; n < n1; ++n) own_end = max(own_end, line.bound(n + 1));
    int run_end = own_end;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int e = __shfl_up_sync(0xffffffffu, run_end, o);
        if (lane >= o) run_end = max(run_end, e);
    }
    if (lane == 31) part_end[warp] = run_end;
    __syncthreads();
    int floor0 = __shfl_up_sync(0xffffffffu, run_end, 1);
    if (lane == 0) floor0 = 0;
    for (int w = 0; w < warp; ++w) floor0 = max(floor0, part_end[w]);
    long long own = 0;
    {
        int f = floor0, b;
        for (int n = n0; n < n1; ++n) own += max(1, (line.length(n, f, b) + C - 1) / C);
    }
    long long run = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long e = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += e;
    }
    if (lane == 31) part[warp] = run;
    __syncthreads();
    long long before = run - own, total = 0;
    for (int w = 0; w < PLAN_THREADS / 32; ++w) {
        if (w < warp) before += part[w];
        total += part[w];
    }
    const long long U = total * H, first = U * blockIdx.x / gridDim.x, end = U * (blockIdx.x + 1) / gridDim.x;
    if (blockIdx.x == 0 && tid == 0) *A.total = U;
    if (first >= end) return;
    {
        long long at = before;
        int f = floor0, b;
        for (int n = n0; n < n1; ++n) {
            const int was = f, chunks = max(1, (line.length(n, f, b) + C - 1) / C);
            const long long u = first - at * H;
            if (u >= 0 && u < (long long)chunks * H) {
                found[0] = n;
                found[1] = (int)(u / chunks);
                found[2] = (int)(u % chunks);
                found[3] = was;
            }
            at += chunks;
        }
    }
    __syncthreads();
    int n = found[0], h = found[1], floor = found[3], begin;
    long long pos = found[2] + warp;
    int len = line.length(n, floor, begin), chunks = max(1, (len + C - 1) / C);
    for (long long u = first + warp; u < end; u += PLAN_THREADS / 32, pos += PLAN_THREADS / 32) {
        while (pos >= chunks) {
            pos -= chunks;
            if (++h == H) {
                h = 0;
                ++n;
                len = line.length(n, floor, begin);
                chunks = max(1, (len + C - 1) / C);
            }
        }
        for (int k = 0; k < A.variants; ++k) {
            const bool reverse = A.reverse[k];
            const int chunk = reverse ? chunks - 1 - (int)pos : (int)pos, t0 = begin + chunk * C, valid = min(C, len - chunk * C);
            Record &R = A.rec[k][u];
            float g[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                g[e] = t < valid ? __ldg(A.g + (A.fixed ? (size_t)h : (size_t)(t0 + t) * H + h)) : 0.f;
            }
            const long long d1 = decay_units(g[1]);
            long long v = decay_units(g[0]) + d1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long e = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += e;
            }
            const long long all = __shfl_sync(0xffffffffu, v, 31);
            const unsigned bad0 = __ballot_sync(0xffffffffu, g[0] != g[0]), bad1 = __ballot_sync(0xffffffffu, g[1] != g[1]);
            unsigned long long bad = 0;
            if (bad0 | bad1)
                for (int i = 0; i < 32; ++i) bad |= (unsigned long long)((bad0 >> i & 1) | (bad1 >> i & 1) << 1) << (2 * i);
            const float nan = __int_as_float(0x7fffffff), sign = reverse ? -1.f : 1.f;
            const float2 whole = two_floats(all);
            bool plain = true;
            float2 x[2];
            float c[2], w[2], fi[2], fj[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const unsigned long long upto = ~0ull >> (63 - 2 * lane - e);
                const float2 f = two_floats(e ? v : v - d1);
                const float up = ex2(f.x) * ex2(f.y), down = ex2(whole.x - f.x) * ex2(whole.y - f.y), inverse = ex2(-f.x) * ex2(-f.y);
                x[e] = make_float2(sign * f.x, sign * f.y);
                c[e] = bad & (reverse ? ~upto : upto) ? nan : A.sc[k] * (reverse ? down : up);
                w[e] = bad & (reverse ? upto : ~upto) ? nan : A.sw[k] * (reverse ? up : down);
                fi[e] = reverse ? inverse : up;
                fj[e] = A.sp[k] * (reverse ? up : inverse);
                plain = plain && fabsf(f.x) < 100.f;
            }
            // (sums of up to 100 powers of two and a scale of up to 2^25 or down to 2^-25: neither factor leaves FP32's range, and their
            // product is D's)
            plain = __all_sync(0xffffffffu, plain) && !bad && fabsf(A.sp[k]) < 33554432.f && fabsf(A.sp[k]) > 2.98e-8f;
            reinterpret_cast<float4 *>(R.g)[lane] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
            reinterpret_cast<float2 *>(R.c)[lane] = make_float2(c[0], c[1]);
            reinterpret_cast<float2 *>(R.w)[lane] = make_float2(w[0], w[1]);
            reinterpret_cast<float2 *>(R.fi)[lane] = make_float2(fi[0], fi[1]);
            reinterpret_cast<float2 *>(R.fj)[lane] = make_float2(fj[0], fj[1]);
            if (lane == 0) {
                R.lost = bad;
                R.units = all;
                R.keep = bad ? nan : ex2(whole.x) * ex2(whole.y);
                R.plain = plain;
                R.n = n;
                R.h = h;
                R.hk = h / A.group;
                R.t0 = t0;
                R.valid = valid;
                R.chunk = chunk;
                R.pos = (int)pos;
                R.chunks = chunks;
            }
        }
    }
}

template <Kind KIND> __global__ void __launch_bounds__(THREADS, 1) tc_kernel(const __grid_constant__ TcArgs A) {
    constexpr bool STATES = KIND == kStates, FULL = KIND == kFull;
    using M = Map<KIND>;
    constexpr int STAGES = M::STAGES, SETS = M::SETS;
    extern __shared__ uint8_t raw[];
    uint8_t *const sm = smem_align1024(raw);
    const uint32_t sm32 = smem_u32(sm);
    Shared &sh = *reinterpret_cast<Shared *>(sm + M::INFO);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int job = blockIdx.x / A.pieces, piece = blockIdx.x % A.pieces;
    const Job &J = A.c.job[job];
    const int H = A.c.H;
    const Waiter wait{&sh.dead};
    const Record *const line = A.rec[job];

    let_next_start();
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), STATES ? 1 + HOLD / 32 : 3);
            sh.dirty[s] = 0;
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sh.drain[s]), 1);
            mbar_init(smem_u32(&sh.acc_full[s]), 2);
            mbar_init(smem_u32(&sh.acc_free[s]), HOLD / 32);
        }
        mbar_init(smem_u32(&sh.pt_full), 1);
        mbar_init(smem_u32(&sh.pt_free), 3);
        mbar_init(smem_u32(&sh.prep_full), PREP / 32);
        mbar_init(smem_u32(&sh.sop_full), HOLD / 32);
        mbar_init(smem_u32(&sh.o1_full), 1);
        mbar_init(smem_u32(&sh.out_full), HOLD / 32);
        fence_mbar_init();
        sh.dead = 0;
    }
    for (int i = tid; i < STAGES * D; i += THREADS) sh.poison[i / D][i % D] = NONE;

    if (warp == 0) {
        tmem_alloc(smem_u32(&sh.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh.tmem;
    auto leave = [&] {
        tc_fence_before();
        __syncthreads();
        if (tid == 0 && sh.dead) atomicOr(A.c.status, 2u);
        if (warp == 0) {
            tc_fence_after();
            tmem_dealloc(tm, 512);
        }
    };
    wait_for_last();

    // ---- where the piece begins and ends
    const long long U = *A.total;
    // (halves are there where each of them has a chunk)
    const int coarse = A.nested ? A.fine / 2 : A.fine;
    const long long most = worth(U, (long long)A.c.N * H, coarse);
    const int count_fine = A.nested && most > coarse && U >= A.fine ? A.fine : (int)min((long long)coarse, most);
    const int halves = FULL && A.pieces != A.fine && count_fine > coarse ? 2 : 1, count_pieces = count_fine / halves;
    if (piece >= count_pieces) {
        if (STATES && tid == 0) A.head[job * A.fine + piece] = Head{0.f, 0, 0};
        return leave();
    }
    long long u0 = U * piece / count_pieces;
    const long long u1 = U * (piece + 1) / count_pieces;
    if constexpr (STATES) {
        const int pos1 = u1 < U ? line[u1].pos : 0;                  // within a pair: its part of this piece, if it ends there
        const bool goes_on = u1 - pos1 < u0;
        if (!goes_on) u0 = u1 - pos1;
        if (tid == 0) {
            Head &hd = A.head[job * A.fine + piece];
            hd.ends_within = pos1 > 0;
            hd.goes_on = pos1 > 0 && goes_on;
        }
        if (pos1 == 0) return leave();
    }
    const int items = (int)(u1 - u0);
    // (in registers: read where they are used, they would be fetched anew from the parameters each time)
    const bool reverse = J.reverse, dots = FULL && J.dots;
    constexpr bool exact = FULL;

    if (warp < PREP_WARP) {
        give_registers<REG_CTL>();
        if (warp == 0) {
            // ---------------- copies ----------------
            const void *mx = &A.map[A.x[job]], *my = &A.map[A.y[job]], *mz = &A.map[A.z[job]], *mr = FULL ? &A.map[A.r[job]] : nullptr;
            const bool sx = J.x.share > 1, sy = J.y.share > 1, sz = J.z.share > 1, sr = FULL && J.r.share > 1;
            const uint32_t bytes = (uint32_t)(STATES ? 4 : FULL && dots ? 8 : 6) * A.rows * 128 + (uint32_t)sizeof(Record);
            int at_t0 = 0, at_h = 0, at_hk = 0;                      // of 32 chunks, one a lane
            int it = 0;
            for (; it < items; ++it) {
                const int s = it % STAGES;
                if (it % 32 == 0) {
                    const Record &R = line[u0 + min(it + lane, items - 1)];
                    at_t0 = R.t0;
                    at_h = R.h;
                    at_hk = R.hk;
                }
                const int t0 = uniform(__shfl_sync(0xffffffffu, at_t0, it & 31)), h = uniform(__shfl_sync(0xffffffffu, at_h, it & 31)),
                          hk = uniform(__shfl_sync(0xffffffffu, at_hk, it & 31));
                if (it >= STAGES) {
                    if (!wait(sh.empty[s], it / STAGES - 1)) break;
                    if (sh.dirty[s]) {
                        for (int i = lane; i < D; i += 32) sh.poison[s][i] = NONE;
                        __syncwarp();
                        sh.dirty[s] = 0;
                    }
                }
                __syncwarp();
                const uint32_t bar = uniform(smem_u32(&sh.full[s])), to = uniform(sm32 + s * M::STAGE), rec_at = uniform(smem_u32(&sh.rec[s]));
                const char *const rec = uniform(reinterpret_cast<const char *>(line + u0 + it));
                if (elect()) {
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_g2s(rec_at, rec, (uint32_t)sizeof(Record), bar);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        tma_load_3d(to + M::Y + u * M::ATOM, my, 64 * u, sy ? hk : h, t0, bar);
                        if (!STATES) tma_load_3d(to + M::XT + u * M::ATOM, mx, 64 * u, sx ? hk : h, t0, bar);
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) tma_load_3d(to + M::Z + u * TILE, mz, 64 * u, sz ? hk : h, t0, bar);
                    if (FULL && dots)
#pragma unroll
                        for (int u = 0; u < 2; ++u) tma_load_3d(to + M::R + u * TILE, mr, 64 * u, sr ? hk : h, t0, bar);
                }
                __syncwarp();
            }
            // (after a wait that gave up: nothing may be on its way into shared memory when the CTA ends)
            for (int k = max(0, it - STAGES); k < it; ++k)
#pragma unroll 1
                for (uint32_t i = 0; i < kTries && !mbar_try_wait(smem_u32(&sh.full[k % STAGES]), (k / STAGES) & 1); ++i) {}
        } else if (warp == 1) {
            // ---------------- products: the chunk's parts of the state and of the outputs ----------------
            const uint32_t tu = uniform(tm), base = uniform(sm32);
            for (int it = 0; it < items; ++it) {
                const int s = it % STAGES, set = it % SETS;
                if (!wait(sh.prep_full, it) || (it >= SETS && !wait(sh.acc_free[set], it / SETS - 1)) || !wait(sh.full[s], it / STAGES)) break;
                tc_fence_after();
                const uint32_t stage = uniform(base + s * M::STAGE), at = uniform(base + M::OPS + set * M::SET), to = uniform(tu + ACC + set * ACC_STEP);
                if (elect()) {
                    constexpr uint32_t wide = idesc_bf16_f32(128, 192, false, true, true), narrow = idesc_bf16_f32(128, 128, false, true, true);
                    const uint64_t z = sdesc_mnmajor_sw128(stage + M::Z, TILE), ops = sdesc_mnmajor_sw128(at, TILE);
                    // parts 1, 2, 0: those of less weight first
#pragma unroll
                    for (int u = 0; u < 3; ++u) {
                        const int p = u == 0 ? 1 : u == 1 ? 2 : 0;
                        const uint32_t id = STATES || (p == 2 && !exact) ? narrow : wide;
#pragma unroll
                        for (int k = 0; k < C / 16; ++k) mma_bf16(to, dadd(z, k * 2048), dadd(ops, p * M::PART + k * 2048), id, u + k > 0);
                    }
                    mma_commit(smem_u32(&sh.acc_full[set]));
                    mbar_arrive(smem_u32(&sh.acc_full[set]));        // (what the preparing warps noted is passed on by a plain arrival)
                    mma_commit(smem_u32(&sh.empty[s]));
                }
                __syncwarp();
            }
            // every product has ended before the CTA does
            if (elect()) mma_commit(smem_u32(&sh.drain[0]));
#pragma unroll 1
            for (uint32_t i = 0; i < kTries && !mbar_try_wait(smem_u32(&sh.drain[0]), 0); ++i) {}
        } else if (!STATES && warp == 2) {
            // ---------------- products: what the state gives; the next chunk's scores ----------------
            const bool wide_a = J.a > 64;
            const uint32_t tu = uniform(tm), base = uniform(sm32);
            constexpr uint32_t id = idesc_bf16_f32(128, 64);
            for (int it = -1; it < items; ++it) {
                if (it + 1 < items) {
                    const int s = (it + 1) % STAGES;
                    if (!wait(sh.full[s], (it + 1) / STAGES) || (it >= 0 && !wait(sh.pt_free, it))) break;
                    tc_fence_after();
                    const uint32_t stage = uniform(base + s * M::STAGE);
                    if (elect()) {
                        const uint64_t y = sdesc_kmajor_sw128(stage + M::Y), x = sdesc_kmajor_sw128(stage + M::XT);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (k < 4 || wide_a)
                                mma_bf16(tu + PT, dadd(y, (k >> 2) * M::ATOM + (k & 3) * 32), dadd(x, (k >> 2) * M::ATOM + (k & 3) * 32), id, k > 0);
                        mma_commit(smem_u32(&sh.pt_full));
                    }
                    __syncwarp();
                }
                if (it >= 0) {
                    const int s = it % STAGES;
                    if (!wait(sh.sop_full, it)) break;
                    tc_fence_after();
                    const uint32_t stage = uniform(base + s * M::STAGE);
                    if (elect()) {
                        const uint64_t x = sdesc_kmajor_sw128(stage + M::XT);
                        if (exact)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (k < 4 || wide_a) mma_bf16_ta(tu + O1, tu + SOP + 128 + k * 8, dadd(x, (k >> 2) * M::ATOM + (k & 3) * 32), id, k > 0);
#pragma unroll
                        for (int p = 1; p >= 0; --p)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (k < 4 || wide_a)
                                    mma_bf16_ta(tu + O1, tu + SOP + p * 64 + k * 8, dadd(x, (k >> 2) * M::ATOM + (k & 3) * 32), id, p == 0 || k > 0 || exact);
                        mma_commit(smem_u32(&sh.o1_full));
                        mma_commit(smem_u32(&sh.empty[s]));
                    }
                    __syncwarp();
                }
            }
            if (elect()) mma_commit(smem_u32(&sh.drain[1]));
#pragma unroll 1
            for (uint32_t i = 0; i < kTries && !mbar_try_wait(smem_u32(&sh.drain[1]), 0); ++i) {}
        } else if (!STATES) {
            // ---------------- rows out ----------------
            const void *const map = &A.out[job];
            const bool copied = J.out_bf16;
            const int jb = J.b;
            for (int it = 0; it < items; ++it) {
                const int s = it % STAGES;
                if (!wait(sh.out_full, it)) break;
                const Record &I = sh.rec[s];
                if (lane == 0) {
                    if (copied && I.valid == C) {
                        const uint32_t at = sm32 + s * M::STAGE + M::XT;
                        tma_store_3d(map, at, 0, I.h, I.t0);
                        if (jb > 64) tma_store_3d(map, at + M::ATOM, 64, I.h, I.t0);
                        bulk_commit();
                        bulk_wait_read_all();
                    }
                    mbar_arrive(smem_u32(&sh.empty[s]));
                }
                __syncwarp();
            }
            if (lane == 0) bulk_wait_all();
        }
    } else if (warp < HOLD_WARP) {
        // ---------------- scores and keys as operands ----------------
        if (REG_PREP < 72) give_registers<REG_PREP>();
        // Both operands are free once the chunk before has been summed.  Until then the scores are worked out into registers (by three
        // warps: one quarter of them is not seen and stays 0), and z is looked through by four; then all write.  The keys are 32 units of 32
        // rows and 8 channels, shared out so that all warps end together.
        const int pw = warp - PREP_WARP, quarter = warp & 3;
        const bool keys = STATES || quarter >= 2;
        const int kw = STATES ? pw : (pw >> 2) * 2 + (quarter & 1);
        // z: row `t` of atom `atom`, pieces from c0; scores: row `t`, columns from `i0`
        const int t = 32 * (kw & 1) + lane, atom = (kw >> 1) & 1, i0 = 32 * atom, c0 = STATES ? (kw >> 2) * 4 : 0;
        const int unseen = reverse ? 1 : 2, block = 2 * (quarter & 1) + atom;            // (blocks: 2 row half + column half)
        const bool zero = !keys && block == unseen;
        const int u0 = STATES ? 4 * pw : keys ? 5 * kw : zero ? 26 : 20 + 2 * (block - (block > unseen)), u1 = u0 + (STATES ? 4 : keys ? 5 : zero ? 6 : 2);
        constexpr int SCAN = STATES ? 4 : 8;                         // pieces of z that a warp looks through
        const float sp = J.sp;
        for (int it = 0; it < items; ++it) {
            const int s = it % STAGES, set = it % SETS;
            uint8_t *const ops = sm + M::OPS + set * M::SET, *const row_at = ops + (uint32_t)t * 128, *const stage = sm + s * M::STAGE;
            if (!wait(sh.full[s], it / STAGES)) break;
            const Record &I = sh.rec[s];
            const int valid = I.valid;
            if (keys) {
                // z: rows behind the sequence are put to 0, and what is not finite, which is noted.  (Piece c of row t lies at piece
                // c ^ (t & 7): the lanes' rows, taken in that order, lie in different banks.)
                uint8_t *const z = stage + M::Z + atom * TILE + (uint32_t)t * 128;
                if (t >= valid) {
#pragma unroll 1
                    for (int c = 0; c < SCAN; ++c) *reinterpret_cast<uint4 *>(z + ((c0 + c) ^ (t & 7)) * 16) = make_uint4(0, 0, 0, 0);
                } else {
                    uint32_t most = 0;
#pragma unroll 2
                    for (int c = 0; c < SCAN; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(z + ((c0 + c) ^ (t & 7)) * 16);
                        most = __vmaxu2(__vmaxu2(most, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu);
                        most = __vmaxu2(__vmaxu2(most, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu);
                    }
                    if ((most & 0xffffu) >= 0x7f80u || most >= 0x7f800000u) {
#pragma unroll 1
                        for (int e = 0; e < SCAN * 8; ++e) {
                            unsigned short *p = reinterpret_cast<unsigned short *>(z + ((c0 + e / 8) ^ (t & 7)) * 16) + e % 8;
                            if ((*p & 0x7fffu) < 0x7f80u) continue;
                            *p = 0;
                            note_first(sh.poison[s], atom * 64 + c0 * 8 + e, reverse ? C - 1 - t : t);
                            sh.dirty[s] = 1;
                        }
                    }
                }
                if (it >= SETS && !wait(sh.acc_full[set], it / SETS - 1)) break;      // the operands' last reader
            } else if (zero) {
                if (it >= SETS && !wait(sh.acc_full[set], it / SETS - 1)) break;
                if (it == 0)
#pragma unroll 1
                    for (int c = 0; c < 12; ++c)
                        if (c < (FULL ? 12 : 8)) *reinterpret_cast<uint4 *>(row_at + 2 * TILE + (c >> 2) * M::PART + (((i0 >> 3) + (c & 3)) ^ (t & 7)) * 16) = make_uint4(0, 0, 0, 0);
            } else if constexpr (!STATES) {
                if (!wait(sh.pt_full, it)) break;
                tc_fence_after();
                // columns that row t is seen by, in the thread's 32, as bits
                const uint32_t lower = 0xffffffffu >> (31 - lane), mask = t >= valid ? 0u : i0 != 32 * quarter ? 0xffffffffu : reverse ? lower : ~(lower >> 1);
                // the diagonal stays out of P where the dots want it so, and is kept
                const uint32_t apart = dots && i0 == 32 * quarter ? 1u << lane : 0u;
                float own = 0.f;
                const float fj = I.fj[t];
                const bool plain = I.plain;
                // columns g to g + 7, in parts
                auto group = [&](int g, uint32_t (&part)[FULL ? 3 : 2][4]) {
                    uint32_t r[8];
                    float p[8];
                    tmem_ld8(tm + ((uint32_t)quarter * 32 << 16) + PT + i0 + g, r);
                    if (plain) {
                        *reinterpret_cast<float4 *>(p) = *reinterpret_cast<const float4 *>(&I.fi[i0 + g]);
                        *reinterpret_cast<float4 *>(p + 4) = *reinterpret_cast<const float4 *>(&I.fi[i0 + g + 4]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) p[e] *= fj;
                    } else {
                        const float2 gj = I.g[t];
                        const unsigned long long lost = I.lost;
#pragma unroll 1
                        for (int e = 0; e < 8; ++e) {
                            const int i = i0 + g + e;
                            const float2 gi = I.g[i];
                            const bool cut = ((~0ull >> (63 - i)) ^ (~0ull >> (63 - t))) & lost;
                            const float v = cut ? __int_as_float(0x7fffffff) : sp * ex2((gi.x - gj.x) + (gi.y - gj.y));
#pragma unroll
                            for (int u = 0; u < 8; ++u)
                                if (u == e) p[u] = v;
                        }
                    }
                    tmem_wait_ld();
                    const uint32_t seen = mask >> g, out = apart >> g;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        p[e] = seen >> e & 1 ? p[e] * __uint_as_float(r[e]) : 0.f;
                        if (FULL) {
                            own = out >> e & 1 ? p[e] : own;
                            p[e] = out >> e & 1 ? 0.f : p[e];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        part[0][e] = peel(p[2 * e], p[2 * e + 1]);
                        if constexpr (FULL) {
                            part[1][e] = peel(p[2 * e], p[2 * e + 1]);
                            part[2][e] = pack(p[2 * e], p[2 * e + 1]);
                        } else {
                            part[1][e] = pack(p[2 * e], p[2 * e + 1]);
                        }
                    }
                };
                auto put = [&](int g, const uint32_t (&part)[FULL ? 3 : 2][4]) {
                    uint8_t *const to = row_at + 2 * TILE + (uint32_t)(((i0 + g) >> 3) ^ (t & 7)) * 16;
#pragma unroll
                    for (int u = 0; u < (FULL ? 3 : 2); ++u) *reinterpret_cast<uint4 *>(to + u * M::PART) = make_uint4(part[u][0], part[u][1], part[u][2], part[u][3]);
                };
                if constexpr (FULL) {
                    // (48 registers of three parts would not do: the copies, two stages deep, are what this waits for anyway)
                    if (it >= SETS && !wait(sh.acc_full[set], it / SETS - 1)) break;
#pragma unroll 1
                    for (int g = 0; g < 32; g += 8) {
                        uint32_t part[FULL ? 3 : 2][4];
                        group(g, part);
                        put(g, part);
                    }
                    if (apart) sh.own[s][t] = own;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_relaxed(sh.pt_free);
                } else {
                    uint32_t part[4][FULL ? 3 : 2][4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) group(8 * g, part[g]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_relaxed(sh.pt_free);
                    if (it >= SETS && !wait(sh.acc_full[set], it / SETS - 1)) break;
#pragma unroll
                    for (int g = 0; g < 4; ++g) put(8 * g, part[g]);
                }
            }
#pragma unroll 1
            for (int u = u0; u < u1; ++u) {
                const int row = 32 * (u >> 3 & 1) + lane, half = u >> 4, at = row * 128 + ((u & 7) ^ (row & 7)) * 16;
                uint4 v = *reinterpret_cast<const uint4 *>(stage + M::Y + half * M::ATOM + at);
                float w = I.w[row];
                if (row >= valid) {
                    v = make_uint4(0, 0, 0, 0);
                    w = 0.f;
                }
                const uint32_t in4[4] = {v.x, v.y, v.z, v.w};
                uint32_t out[3][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float a = low(in4[e]) * w, b = high(in4[e]) * w;
                    out[0][e] = peel(a, b);
                    out[1][e] = peel(a, b);
                    out[2][e] = pack(a, b);
                }
#pragma unroll
                for (int e = 0; e < 3; ++e) *reinterpret_cast<uint4 *>(ops + half * TILE + e * M::PART + at) = make_uint4(out[e][0], out[e][1], out[e][2], out[e][3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.prep_full));
        }
    } else {
        // ---------------- the state, and what is put out ----------------
        take_registers<REG_HOLD>();
        const int hw = warp - HOLD_WARP, part = hw >> 2, b = 32 * (warp & 3) + lane, a0 = COLS * part;
        const uint32_t lanes = tm + ((uint32_t)(warp & 3) * 32 << 16);
        const int ja = J.a, jb = J.b, sa = J.sa, sb = J.sb;
        const bool in_b = b < jb, out_bf16 = J.out_bf16;
        const float *const first = J.first;
        float *const last = J.last, *const anchors = FULL ? J.anchors : nullptr, *const dots_at = J.dots;
        const bool last_anchor = J.last_anchor;
        char *const out = static_cast<char *>(J.out);
        const uint32_t row_step = (uint32_t)H * jb * (FULL && !out_bf16 ? 4 : 2);
        float S[COLS];
#pragma unroll
        for (int i = 0; i < COLS; ++i) S[i] = 0.f;
        float *const own_state = A.state + ((size_t)job * A.fine + piece) * D * D;       // (states)
        const bool turned = FULL && A.turned[job];
        // the state that chunk `it` begins with
        auto enter = [&](int it) {
            const Record &I = sh.rec[it % STAGES];
            const bool begins = I.pos == 0, open = begins && I.chunks > items - it;      // open: the pair ends in another piece
            if (!begins && it > 0) return;
            const int slot = seq_slot(A.c.slot, A.c.num_slots, I.n);
            const size_t state = ((size_t)max(slot, 0) * H + I.h) * ja * jb;
            // element a of it is at from[a * step]; nothing (zero) without one
            const float *from = begins ? (first && slot >= 0 && in_b ? first + state + (size_t)b * sb : nullptr)
                                                   : (STATES ? nullptr : A.state + ((size_t)A.of[job] * A.fine + piece * halves - 1) * D * D + (turned ? b * D : b));
            int step = begins ? sa : turned ? 1 : D;
            if (A.kept && open) {
                float *const kept = A.kept + (size_t)piece * D * D + b;
                if (STATES) {
#pragma unroll 4
                    for (int i = a0; i < min(ja, a0 + COLS); ++i) kept[(size_t)i * D] = from ? from[(size_t)i * step] : 0.f;
                } else {
                    from = kept;
                    step = D;
                }
            }
            if (from) from += (size_t)a0 * step;
            const int rows = from ? ja - a0 : 0;
#pragma unroll
            for (int i = 0; i < COLS; ++i) {
                S[i] = i < rows ? *from : 0.f;
                from += step;
            }
        };
        // S as an operand: a pair of columns a word
        auto hand_over = [&] {
#pragma unroll
            for (int q = 0; q < COLS / 16; ++q) {
                uint32_t w[3][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float x = S[16 * q + 2 * i], y = S[16 * q + 2 * i + 1];
                    w[0][i] = peel(x, y);
                    if (exact) {
                        w[1][i] = peel(x, y);
                        w[2][i] = pack(x, y);
                    } else {
                        w[1][i] = pack(x, y);
                    }
                }
                tmem_st8(lanes + SOP + a0 / 2 + 8 * q, w[0]);
                tmem_st8(lanes + SOP + 64 + a0 / 2 + 8 * q, w[1]);
                if (exact) tmem_st8(lanes + SOP + 128 + a0 / 2 + 8 * q, w[2]);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_relaxed(sh.sop_full);
        };
        bool ok = true, lost = false;
        long long units = 0;                                         // STATES: the piece's decay
        for (int it = -1; it < items; ++it) {                        // (-1: only the first state goes out)
            const int set = it & (SETS - 1);
            const uint32_t acc = lanes + ACC + set * ACC_STEP;
            const int s = it < 0 ? 0 : it % STAGES;
            const Record &I = sh.rec[s];
            bool ends = false;
            int n = 0, h = 0, t0 = 0, valid = 0, chunk = 0;
            bool dirty = false;
            float o[TOKENS];
            if (it >= 0) ok = ok && wait(sh.acc_full[set], it / SETS);
            if (ok && it >= 0) {
                tc_fence_after();
                ends = I.pos == I.chunks - 1;
                n = I.n;
                h = I.h;
                t0 = I.t0;
                valid = I.valid;
                chunk = I.chunk;
                dirty = sh.dirty[s];
                if (STATES) {
                    units = add_units(units, I.units);
                    lost = lost || I.lost;
                }
                const float keep = I.keep;
                const int poison = dirty ? sh.poison[s][b] : NONE;
#pragma unroll
                for (int q = 0; q < COLS / 16; ++q) {
                    uint32_t r[16];
                    tmem_ld16(acc + a0 + 16 * q, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) S[16 * q + i] = fmaf(keep, S[16 * q + i], __uint_as_float(r[i]));
                }
                if (poison != NONE)
#pragma unroll
                    for (int i = 0; i < COLS; ++i) S[i] = __int_as_float(0x7fffffff);
                if constexpr (!STATES) {
                    uint32_t r[16];
                    tmem_ld16(lanes + ACC_O + TOKENS * part, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __uint_as_float(r[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_relaxed(sh.acc_free[set]);
                if constexpr (!STATES) {
                    ok = wait(sh.o1_full, it);
                    if (ok) {
                        tc_fence_after();
                        uint32_t r[16];
                        tmem_ld16(lanes + O1 + TOKENS * part, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 c = *reinterpret_cast<const float4 *>(&I.c[TOKENS * part + i]);
                            o[i] = fmaf(c.x, __uint_as_float(r[i]), o[i]);
                            o[i + 1] = fmaf(c.y, __uint_as_float(r[i + 1]), o[i + 1]);
                            o[i + 2] = fmaf(c.z, __uint_as_float(r[i + 2]), o[i + 2]);
                            o[i + 3] = fmaf(c.w, __uint_as_float(r[i + 3]), o[i + 3]);
                        }
                        if (poison != NONE)
#pragma unroll
                            for (int i = 0; i < TOKENS; ++i)
                                if ((reverse ? C - 1 - TOKENS * part - i : TOKENS * part + i) >= poison) o[i] = __int_as_float(0x7fffffff);
                    }
                }
            }
            if (!ok) break;
            if (STATES) {
                __syncwarp();
                if (it >= 0 && lane == 0) mbar_arrive(smem_u32(&sh.empty[s]));
            } else if (it >= 0) {
                // where channel b of a token stands in a tile: piece (b / 8) ^ (token & 7) of the token's row
                const uint32_t tile = (b >> 6) * TILE + part * TOKENS * 128 + (b & 7) * 2;
                uint8_t *const stage = sm + s * M::STAGE;
                float d[FULL ? TOKENS : 1];
                if (FULL && dots) {
                    // the dots of the warp's channels, and the term of the token itself, which is in the rows but not in them
                    const int left = in_b ? valid - TOKENS * part : 0;
                    float4 own;
#pragma unroll
                    for (int i = 0; i < TOKENS; ++i) {
                        if (i % 4 == 0) own = *reinterpret_cast<const float4 *>(&sh.own[s][TOKENS * part + i]);
                        const uint32_t at = tile + i * 128 + (((b >> 3) ^ i) & 7) * 16;
                        const unsigned short r = *reinterpret_cast<const unsigned short *>(stage + M::R + at), z = *reinterpret_cast<const unsigned short *>(stage + M::Z + at);
                        d[i] = i < left ? __uint_as_float((uint32_t)r << 16) * o[i] : 0.f;
                        o[i] = fmaf(i % 4 == 0 ? own.x : i % 4 == 1 ? own.y : i % 4 == 2 ? own.z : own.w, __uint_as_float((uint32_t)z << 16), o[i]);
                    }
                }
                if (valid == C && (!FULL || out_bf16)) {
                    // (x, in whose place they go, has been used)
                    uint8_t *const x = stage + M::XT + (b >> 6) * (M::ATOM - TILE) + tile;
#pragma unroll
                    for (int i = 0; i < TOKENS; ++i) *reinterpret_cast<__nv_bfloat16 *>(x + i * 128 + (((b >> 3) ^ i) & 7) * 16) = __float2bfloat16_rn(o[i]);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.out_full));
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.out_full));          // (an arrival behind the stores would wait for them)
                    // a channel a lane, a token a store; one address for the warp and 32-bit offsets
                    const int left = in_b ? valid - TOKENS * part : 0;
                    char *const rows = uniform(out + ((size_t)(t0 + TOKENS * part) * H + h) * jb * (FULL && !out_bf16 ? 4 : 2));
                    if (FULL && !out_bf16) {
#pragma unroll
                        for (int i = 0; i < TOKENS; ++i) store_if(i < left, rows + (4 * b + i * row_step), o[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < TOKENS; ++i) store_if(i < left, rows + (2 * b + i * row_step), __float2bfloat16_rn(o[i]));
                    }
                }
                if (FULL && dots) {
                    // sums over the lanes, half of the tokens given away at each step
#pragma unroll
                    for (int w = 8; w; w >>= 1)
#pragma unroll
                        for (int i = 0; i < w; ++i) {
                            const bool upper = lane & 2 * w;
                            const float give = upper ? d[i] : d[i + w], keep = upper ? d[i + w] : d[i];
                            d[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * w);
                        }
                    d[0] += __shfl_xor_sync(0xffffffffu, d[0], 1);
                    const int t = TOKENS * part + (lane >> 1);
                    if (!(lane & 1) && t < valid) dots_at[((size_t)(warp & 3) * A.c.T + t0 + t) * H + h] = d[0];
                }
            }
            {
                // where the state goes: to an anchor, to the caller, to the piece that goes on
                const int behind = reverse ? chunk * C : chunk * C + valid, begin = t0 - chunk * C;
                const bool at_anchor = anchors && it >= 0 && (ends ? last_anchor : behind % kAnchor == 0);
                const bool to_last = !STATES && ends && last, to_piece = STATES && it == items - 1;
                if (at_anchor || to_last || to_piece) {
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        float *to = nullptr;
                        int step = 0;
                        if (k == 0 && at_anchor) {
                            // (the last state has the sequence's last slot; its record is read again: the stage may have been given away)
                            const int stretch = ends ? (line[u0 + it].chunks - 1) / (kAnchor / C) : (behind - 1) / kAnchor;
                            to = anchors + ((size_t)(anchor_slot(begin, n) + stretch) * H + h) * ja * jb + b;
                            step = jb;
                        }
                        if (k == 1 && to_last) {
                            const int slot = seq_slot(A.c.slot, A.c.num_slots, n);
                            if (slot >= 0) to = last + ((size_t)slot * H + h) * ja * jb + (size_t)b * sb;
                            step = sa;
                        }
                        if (k == 1 && to_piece) {
                            to = own_state + b;
                            step = D;
                        }
                        if (!to || !(in_b || STATES)) continue;
                        const int rows = (STATES ? D : ja) - a0;
                        to += (size_t)a0 * step;
#pragma unroll
                        for (int i = 0; i < COLS; ++i) {
                            if (i < rows) *to = S[i];
                            to += step;
                        }
                    }
                }
                if (it + 1 < items) {
                    ok = wait(sh.full[(it + 1) % STAGES], (it + 1) / STAGES);
                    if (ok) {
                        enter(it + 1);
                        if (!STATES) hand_over();
                    }
                }
            }
        }
        if (STATES && threadIdx.x == CTL + PREP) A.head[job * A.fine + piece].keep = lost ? __int_as_float(0x7fffffff) : exp2_units(units);
    }
    leave();
}

// The states that pieces leave, one after the other within a pair: S_piece += decay_piece S_before, from the piece that holds the pair's
// start on.  A CTA a slice of the state and first piece; 7 us, a launch's start and three loads in turn.
__global__ void __launch_bounds__(256) join_kernel(const Head *head, float *state, int pieces) {
    let_next_start();
    wait_for_last();
    head += (size_t)blockIdx.z * pieces;
    state += ((size_t)blockIdx.z * pieces) * D * D + (size_t)blockIdx.x * 1024 + threadIdx.x * 4;
    int c = blockIdx.y;
    if (!head[c].ends_within || head[c].goes_on) return;
    float4 v = *reinterpret_cast<float4 *>(state + (size_t)c * D * D);
    for (++c; c < pieces && head[c].ends_within && head[c].goes_on; ++c) {
        float4 *at = reinterpret_cast<float4 *>(state + (size_t)c * D * D);
        const float k = head[c].keep;
        const float4 w = *at;
        v = make_float4(fmaf(k, v.x, w.x), fmaf(k, v.y, w.y), fmaf(k, v.z, w.z), fmaf(k, v.w, w.w));
        *at = v;
    }
}

std::atomic<PFN_cuTensorMapEncodeTiled_v12000> g_encode{nullptr};
std::atomic<uint64_t> g_attr[3];

// [T, heads, d] BF16 in boxes of 64 channels of one head and `rows` tokens; channels and tokens outside read 0.
cudaError_t make_map(CUtensorMap *m, const void *base, int T, int heads, int d, int rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = g_encode.load(std::memory_order_acquire);
    if (!encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) return e != cudaSuccess ? e : cudaErrorSymbolNotFound;
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        g_encode.store(encode, std::memory_order_release);
    }
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
    const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)rows}, ones[3] = {1u, 1u, 1u};
    const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, ones,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A launch, as the one before's programmatic dependent or behind all of it; its error is returned and not left to the next call.
template <class... P, class... X> cudaError_t follow(bool dependent, void (*kernel)(P...), dim3 grid, int threads, size_t bytes, cudaStream_t s, const X &...args) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = bytes;
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = dependent;
    count_launch();
    const cudaError_t e = cudaLaunchKernelEx(&c, kernel, P(args)...);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

}  // namespace

// The pieces' states (of two jobs, or of one with the first states that it keeps) and heads, the number of records, and the records of up
// to two directions.
static size_t states_part() { return (size_t)2 * MOST_PIECES * (D * D * sizeof(float) + sizeof(Head)); }
static size_t fixed_part() { return (states_part() + 8 + 255) & ~size_t(255); }
static size_t records(int N, int T, int H) { return ((size_t)T / C + N) * H * sizeof(Record); }
size_t tc_workspace(int N, int T, int H, int directions) { return fixed_part() + records(N, T, H) * directions; }

// The arguments of a launch for a call's jobs; `pieces` CTAs a job.
static cudaError_t arguments(TcArgs &A, const Call &c, const Record *const *rec, int pieces, int fine) {
    A = TcArgs{};
    A.c = c;
    A.rows = c.T < C ? (c.T < 1 ? 1 : c.T) : C;
    // (arrays may lie in one place with other widths: q, k and v as views of the same memory)
    int maps = 0, width[4] = {};
    Rows of[4] = {};
    for (int j = 0; j < c.jobs; ++j) {
        const Rows *rows[4] = {&c.job[j].x, &c.job[j].y, &c.job[j].z, &c.job[j].r};
        int *at[4] = {&A.x[j], &A.y[j], &A.z[j], &A.r[j]};
        for (int u = 0; u < (c.job[j].dots ? 4 : 3); ++u) {
            const int d = u >= 2 ? c.job[j].b : c.job[j].a;
            int m = 0;
            while (m < maps && (of[m].p != rows[u]->p || of[m].share != rows[u]->share || width[m] != d)) ++m;
            if (m == maps) {
                of[maps] = *rows[u];
                width[maps++] = d;
                if (cudaError_t e = make_map(&A.map[m], rows[u]->p, c.T, c.H / rows[u]->share, d, A.rows)) return e;
            }
            *at[u] = m;
        }
        if (c.job[j].out_bf16)
            if (cudaError_t e = make_map(&A.out[j], c.job[j].out, c.T, c.H, c.job[j].b, A.rows)) return e;
        A.rec[j] = rec[j];
        A.of[j] = j;
    }
    A.pieces = pieces;
    A.fine = fine;
    A.state = static_cast<float *>(c.pieces);
    A.head = reinterpret_cast<Head *>(A.state + (size_t)2 * MOST_PIECES * D * D);
    A.total = reinterpret_cast<long long *>(static_cast<char *>(c.pieces) + states_part());
    if (c.jobs == 1 && c.job[0].first && c.job[0].first == c.job[0].last) A.kept = A.state + (size_t)MOST_PIECES * D * D;
    return cudaSuccess;
}

static cudaError_t states(const TcArgs &A, cudaStream_t s) {
    if (cudaError_t e = follow(true, tc_kernel<kStates>, dim3(A.pieces * A.c.jobs), THREADS, kSmem<kStates>, s, A)) return e;
    return follow(true, join_kernel, dim3(D * D / 1024, A.pieces, A.c.jobs), 256, 0, s, A.head, A.state, A.pieces);
}
static cudaError_t outputs(const TcArgs &A, cudaStream_t s) {
    bool plain = true;
    for (int j = 0; j < A.c.jobs; ++j) {
        const Job &b = A.c.job[j];
        plain = plain && b.out_bf16 && !b.exact && !b.dots && !b.anchors;
    }
    return plain ? follow(true, tc_kernel<kPlain>, dim3(A.pieces * A.c.jobs), THREADS, kSmem<kPlain>, s, A)
                 : follow(true, tc_kernel<kFull>, dim3(A.pieces * A.c.jobs), THREADS, kSmem<kFull>, s, A);
}

// The records for some jobs: `rec` gets each one's.
static cudaError_t plan(const Call &c, int sms, const Record **rec, cudaStream_t s) {
    PlanArgs P{};
    P.g = c.g;
    P.cu = c.cu;
    P.fixed = c.fixed;
    P.N = c.N;
    P.T = c.T;
    P.H = c.H;
    P.group = 1;
    P.total = reinterpret_cast<long long *>(static_cast<char *>(c.pieces) + states_part());
    for (int j = 0; j < c.jobs; ++j) {
        const Job &b = c.job[j];
        for (const Rows *r : {&b.x, &b.y, &b.z})
            if (r->share > P.group) P.group = r->share;
        int k = 0;
        while (k < P.variants && (P.reverse[k] != b.reverse || P.sp[k] != b.sp || P.sc[k] != b.sc || P.sw[k] != b.sw)) ++k;
        if (k == P.variants) {
            P.reverse[k] = b.reverse;
            P.sp[k] = b.sp;
            P.sc[k] = b.sc;
            P.sw[k] = b.sw;
            P.rec[k] = reinterpret_cast<Record *>(static_cast<char *>(c.pieces) + fixed_part() + k * records(c.N, c.T, c.H));
            ++P.variants;
        }
        rec[j] = P.rec[k];
    }
    return follow(false, plan_kernel, dim3(2 * sms), PLAN_THREADS, 0, s, P);
}

cudaError_t launch_scan_tc(const Call &c, bool apart, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = smem_attr_once((const void *)tc_kernel<kStates>, (int)kSmem<kStates>, g_attr[0]);
    if (e == cudaSuccess) e = smem_attr_once((const void *)tc_kernel<kPlain>, (int)kSmem<kPlain>, g_attr[1]);
    if (e == cudaSuccess) e = smem_attr_once((const void *)tc_kernel<kFull>, (int)kSmem<kFull>, g_attr[2]);
    if (e != cudaSuccess) return e;
    if (sms > MOST_PIECES) sms = MOST_PIECES;
    const Record *rec[3];
    if (!apart) {
        TcArgs A;
        if ((e = plan(c, sms, rec, s)) != cudaSuccess) return e;          // (the records are addresses to the others)
        if ((e = arguments(A, c, rec, sms / c.jobs, sms / c.jobs)) != cudaSuccess) return e;
        // one short sequence: every piece is a whole pair
        const bool whole = c.N == 1 && (c.T + C - 1) / C < WHOLE && c.H <= A.pieces;
        if (!whole && (e = states(A, s)) != cudaSuccess) return e;
        return outputs(A, s);
    }
    // dq and dv, whose dots and anchors take the operands in three parts, and dk by itself: its rows are all that it puts out.  dv's state is
    // dk's turned, so states are taken for dq and dk, each in as many pieces as dk's launch has; dq's and dv's pieces are two of them.  (8 k
    // tokens and 32 heads: 84 us of states, 123 with those of all three; dk 83, dq and dv 304.)
    const int fine = sms & ~1;
    if ((e = plan(c, sms, rec, s)) != cudaSuccess) return e;
    Call two = c, one = c;
    const Record *rec_two[2] = {rec[0], rec[2]}, *rec_one[1] = {rec[2]};
    two.jobs = 2;
    two.job[1] = c.job[2];
    one.jobs = 1;
    one.job[0] = c.job[2];
    TcArgs A;
    if ((e = arguments(A, two, rec_two, fine, fine)) != cudaSuccess) return e;
    A.nested = true;
    if ((e = states(A, s)) != cudaSuccess) return e;
    if ((e = arguments(A, one, rec_one, fine, fine)) != cudaSuccess) return e;
    A.nested = true;
    A.of[0] = 1;
    if ((e = outputs(A, s)) != cudaSuccess) return e;
    two.job[1] = c.job[1];
    rec_two[1] = rec[1];
    if ((e = arguments(A, two, rec_two, fine / 2, fine)) != cudaSuccess) return e;
    A.nested = A.turned[1] = true;
    return outputs(A, s);
}

}  // namespace lin
}  // namespace k3kda
