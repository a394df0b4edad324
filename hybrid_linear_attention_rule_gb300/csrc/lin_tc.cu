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
// Roles of a CTA, joined by mbarriers: a warp that walks the chunks and sums their decays, ahead of the others; a copy warp (TMA); an MMA
// warp for PT and ACC and one for O1, so that neither chain waits for the other's operands; eight warps that prepare P and
// Yw, sixteen that hold S, write its operand, fold ACC into it and put out rows.
//
// The chunks of all (sequence, head) pairs stand in one line, cut evenly over the CTAs ("pieces").  A piece that begins within a pair
// needs the state there: a first pass (STATES) runs the pieces that end within a pair for their state alone, `join_kernel` chains
// those of a pair, and the second pass starts from them.  The decay of a piece is one number a head, so the chain is a sum.
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

enum Kind { kStates, kPlain, kFull };      // states alone; jobs whose operands are in two parts and that put out nothing but BF16 rows; any, in three parts

constexpr uint32_t TILE = C * 128;                                 // 64 rows of 64 BF16 values
// Shared memory: a ring of copies (y0 [x0] y1 [x1] z0 z1), parts of [Yw0 | Yw1 | P] (twice for the states, whose products then have no gap).
template <Kind K> struct Map {
    static constexpr bool X = K != kStates;
    static constexpr int STAGES = 3, SETS = K == kStates ? 2 : 1;
    static constexpr uint32_t Y = 0, XT = TILE, ATOM = (X ? 2 : 1) * TILE, Z = 2 * ATOM, STAGE = Z + 2 * TILE;
    static constexpr uint32_t OPS = STAGES * STAGE, PART = (X ? 3 : 2) * TILE, SET = K == kPlain ? 2 * PART + 2 * TILE : 3 * PART;
    static constexpr uint32_t INFO = OPS + SETS * SET;
};

struct Item {
    int n, h, hk, t0, valid, chunk, flags;      // hk: h / group
};
struct Place {                 // a chunk on the way to its Info
    float g[C];
    Item item;
};
constexpr int AHEAD = 4, PLACES = 6;
struct alignas(16) Info {      // of one chunk; its arrays are read in 16-byte pieces
    float2 g[C];               // sums of the decays, as two floats; negative backward in time, so that d = g_i - g_j either way
    float c[C], w[C];
    float fi[C], fj[C];        // D_ij = fi[i] fj[j], the scale in fj, where the chunk's decay leaves both in range (`plain`)
    float own[C];              // P's diagonal, where it is kept apart
    float keep;                // the chunk's decay
    unsigned long long lost;   // tokens whose decay is NaN
    Item item;
    int plain;
    int dirty;                 // some z is not finite:
    unsigned char poison[D];   // the channel's first such token in the job's direction, or NONE
};
constexpr int NONE = 255, INFOS = 4;
enum { kFromFirst = 1, kFromPiece = 2, kEnds = 4, kOpen = 8 };        // kOpen: the pair begins here and ends in another piece

struct Shared {
    Info info[INFOS];
    Place place[PLACES];
    unsigned long long info_full[INFOS], info_free[INFOS], full[3], empty[3], pt_full, pt_free, prep_full, acc_full[2], acc_free[2], sop_full, o1_full, drain[2];
    uint32_t tmem;
    int dead;
    long long part[THREADS / 32];
    int part_end[THREADS / 32];
    int n[2], h[2], pos[2], chunks[2], begin[2], len[2], floor[2];     // where the piece begins, and where it ends
};
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
    int x[3], y[3], z[3];      // the jobs' maps
    int rows;                  // of a copy's box
    int group;                 // value heads that share a key head
    int pieces;                // a job
    int least;                 // chunks of a piece, at least, where there are more pieces than pairs
    Head *head;                // [jobs][pieces]
    float *state;              // [jobs][pieces][a][D]
    float *kept;               // likewise, or null: the first states of the pairs that a piece leaves open, when they may be written over
};

template <int N> __device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Stores and loads under a predicate, without a branch around each.
__device__ __forceinline__ void store_if(bool on, char *to, __nv_bfloat16 v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.b16 [%0], %1;\n\t}" ::"l"(to), "h"(__bfloat16_as_ushort(v)), "r"((int)on) : "memory");
}
__device__ __forceinline__ void store_if(bool on, char *to, float v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.f32 [%0], %1;\n\t}" ::"l"(to), "f"(v), "r"((int)on) : "memory");
}
__device__ __forceinline__ float load_bf16_if(bool on, const char *from) {
    unsigned short v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t@p ld.global.nc.b16 %0, [%1];\n\t}" : "=h"(v) : "l"(from), "r"((int)on));
    return __uint_as_float((uint32_t)v << 16);
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
};

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
    const int N = A.c.N, H = A.c.H;
    const Waiter wait{&sh.dead};

    // ---- where the piece begins and ends
    const int per = (N + THREADS - 1) / THREADS, n0 = min(N, tid * per), n1 = min(N, n0 + per);
    const Line line{A.c.cu, A.c.T};
    auto length = [&](int n, int &floor, int &begin) {               // of sequence n; floor: the ends before it
        if (!line.cu) {
            begin = 0;
            return A.c.T;
        }
        begin = max(line.bound(n), floor);
        floor = max(floor, line.bound(n + 1));
        return floor - begin;
    };
    int own_end = 0;
    if (line.cu)
#pragma unroll 1
        for (int n = n0; n < n1; ++n) own_end = max(own_end, line.bound(n + 1));
    int run_end = own_end;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int e = __shfl_up_sync(0xffffffffu, run_end, o);
        if (lane >= o) run_end = max(run_end, e);
    }
    if (lane == 31) sh.part_end[warp] = run_end;
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), (STATES ? 1 : 2) + (FULL && J.dots ? HOLD / 32 : 0));    // (for dots the holding warps read z)
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sh.drain[s]), 1);
            mbar_init(smem_u32(&sh.acc_full[s]), 2);
            mbar_init(smem_u32(&sh.acc_free[s]), HOLD / 32);
        }
        for (int i = 0; i < INFOS; ++i) {
            mbar_init(smem_u32(&sh.info_full[i]), 1);
            mbar_init(smem_u32(&sh.info_free[i]), HOLD / 32);
            sh.info[i].dirty = 0;
        }
        mbar_init(smem_u32(&sh.pt_full), 1);
        mbar_init(smem_u32(&sh.pt_free), 3);
        mbar_init(smem_u32(&sh.prep_full), PREP / 32);
        mbar_init(smem_u32(&sh.sop_full), HOLD / 32);
        mbar_init(smem_u32(&sh.o1_full), 1);
        fence_mbar_init();
        sh.dead = 0;
    }
    for (int i = tid; i < INFOS * D; i += THREADS) sh.info[i / D].poison[i % D] = NONE;
    __syncthreads();
    int floor0 = __shfl_up_sync(0xffffffffu, run_end, 1);
    if (lane == 0) floor0 = 0;
#pragma unroll 1
    for (int w = 0; w < warp; ++w) floor0 = max(floor0, sh.part_end[w]);
    long long own = 0;
    {
        int f = floor0, b;
#pragma unroll 1
        for (int n = n0; n < n1; ++n) own += max(1, (length(n, f, b) + C - 1) / C);
    }
    long long run = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long e = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += e;
    }
    if (lane == 31) sh.part[warp] = run;
    __syncthreads();
    long long before = run - own, total = 0;
#pragma unroll 1
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sh.part[w];
        total += sh.part[w];
    }
    const long long U = total * H, most = max((long long)N * H, U / A.least);
    const int count_pieces = (int)min((long long)A.pieces, most);
    if (piece >= count_pieces) {
        if (STATES && tid == 0) A.head[job * A.pieces + piece] = Head{0.f, 0, 0};
        return;
    }
    long long u0 = U * piece / count_pieces;
    const long long u1 = U * (piece + 1) / count_pieces;
    {
        long long at = before;
        int f = floor0, b;
#pragma unroll 1
        for (int n = n0; n < n1; ++n) {
            const int f_was = f, len = length(n, f, b), chunks = max(1, (len + C - 1) / C);
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
                const long long u = (e ? u1 : u0) - at * H;
                if (u < 0 || u >= (long long)chunks * H) continue;
                sh.n[e] = n;
                sh.h[e] = (int)(u / chunks);
                sh.pos[e] = (int)(u % chunks);
                sh.chunks[e] = chunks;
                sh.begin[e] = b;
                sh.len[e] = len;
                sh.floor[e] = f_was;
            }
            at += chunks;
        }
    }
    __syncthreads();
    int start = 0;                                                   // which of the two places the work begins at
    bool goes_on = false;
    if constexpr (STATES) {
        const bool within = u1 < U && sh.pos[1] > 0;
        if (within) {
            goes_on = u1 - sh.pos[1] < u0;
            if (!goes_on) {
                u0 = u1 - sh.pos[1];
                start = 1;
            }
        }
        if (tid == 0) {
            Head &hd = A.head[job * A.pieces + piece];
            hd.ends_within = within;
            hd.goes_on = goes_on;
        }
        if (!within) return;
    }
    const int items = (int)(u1 - u0);
    const int pos0 = STATES && start == 1 ? 0 : sh.pos[start];

    if (warp == 0) {
        tmem_alloc(smem_u32(&sh.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh.tmem;
    // (in registers: read where they are used, they would be fetched anew from the parameters each time)
    const bool reverse = J.reverse, dots = FULL && J.dots;
    constexpr bool exact = FULL;

    if (warp < PREP_WARP) {
        give_registers<REG_CTL>();
        if (warp == 0) {
            // ---------------- chunks and their decays ----------------
            int n = sh.n[start], h = sh.h[start], pos = pos0, chunks = sh.chunks[start], begin = sh.begin[start], len = sh.len[start];
            int floor = sh.floor[start];
            {
                int b;
                length(n, floor, b);
            }
            int hk = h / A.group, left = A.group - (h - hk * A.group);       // left: heads that still share hk
            long long sum = 0;                                       // STATES: the whole piece's decay
            bool sum_lost = false;
            const float *const g_at = A.c.g;
            const int fixed = A.c.fixed;
            const float sc = J.sc, sw = J.sw, sp = J.sp;
            // (a chunk's decays are a word of every row of g: on their way while those of the chunks before are summed)
            for (int it = -AHEAD; it < items; ++it) {
                const int at = it + AHEAD;
                if (at < items) {
                    if (at > 0 && ++pos == chunks) {
                        pos = 0;
                        if (--left == 0) {
                            left = A.group;
                            ++hk;
                        }
                        if (++h == H) {
                            h = hk = 0;
                            ++n;
                            len = length(n, floor, begin);
                            chunks = max(1, (len + C - 1) / C);
                        }
                    }
                    const int chunk = reverse ? chunks - 1 - pos : pos, t0 = begin + chunk * C, valid = min(C, len - chunk * C);
                    Place &P = sh.place[at % PLACES];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int t = 2 * lane + u;
                        const bool in = t < valid;
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(&P.g[t])), "l"(g_at + (fixed ? (size_t)h : in ? (size_t)(t0 + t) * H + h : 0)),
                                     "r"(in ? 4 : 0)
                                     : "memory");
                    }
                    if (lane == 0)
                        P.item = Item{n, h, hk, t0, valid, chunk, (pos == 0 ? kFromFirst : at == 0 ? kFromPiece : 0) | (pos == chunks - 1 ? kEnds : 0) |
                                                                     (pos == 0 && chunks > items - at ? kOpen : 0)};
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (it < 0) continue;
                asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
                __syncwarp();
                Info &I = sh.info[it % INFOS];
                const Place &P = sh.place[it % PLACES];
                const float g[2] = {P.g[2 * lane], P.g[2 * lane + 1]};
                const long long d0 = decay_units(g[0]), d1 = decay_units(g[1]);
                long long v = d0 + d1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long e = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += e;
                }
                const long long all = __shfl_sync(0xffffffffu, v, 31);
                const unsigned bad0 = __ballot_sync(0xffffffffu, g[0] != g[0]), bad1 = __ballot_sync(0xffffffffu, g[1] != g[1]);
                unsigned long long bad = 0;
                if (bad0 | bad1)
#pragma unroll 1
                    for (int i = 0; i < 32; ++i) bad |= (unsigned long long)((bad0 >> i & 1) | (bad1 >> i & 1) << 1) << (2 * i);
                const float2 whole = two_floats(all);
                const float sign = reverse ? -1.f : 1.f;
                bool plain = true;
                if (it >= INFOS) {
                    if (!wait(sh.info_free[it % INFOS], it / INFOS - 1)) break;
                    if (I.dirty) {
#pragma unroll 1
                        for (int i = lane; i < D; i += 32) I.poison[i] = NONE;
                        __syncwarp();
                        I.dirty = 0;
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = 2 * lane + u;
                    const float2 f = two_floats(u ? v : v - d1);
                    const float up = ex2(f.x) * ex2(f.y), down = ex2(whole.x - f.x) * ex2(whole.y - f.y), inverse = ex2(-f.x) * ex2(-f.y);
                    I.g[t] = make_float2(sign * f.x, sign * f.y);
                    I.c[t] = sc * (reverse ? down : up);
                    I.w[t] = sw * (reverse ? up : down);
                    I.fi[t] = reverse ? inverse : up;
                    I.fj[t] = sp * (reverse ? up : inverse);
                    plain = plain && fabsf(f.x) < 100.f;
                }
                // (sums of up to 100 powers of two: neither factor leaves FP32's range, and their product is D's)
                plain = __all_sync(0xffffffffu, plain) && !bad;
                const float nan = __int_as_float(0x7fffffff);
                if (bad)
#pragma unroll 1
                    for (int t = 2 * lane; t < 2 * lane + 2; ++t) {
                        const unsigned long long upto = ~0ull >> (63 - t);
                        if (bad & (reverse ? ~upto : upto)) I.c[t] = nan;
                        if (bad & (reverse ? upto : ~upto)) I.w[t] = nan;
                    }
                sum += all;
                sum_lost = sum_lost || bad;
                if (lane == 0) {
                    I.keep = bad ? nan : ex2(whole.x) * ex2(whole.y);
                    I.plain = plain;
                    I.lost = bad;
                    I.item = P.item;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.info_full[it % INFOS]));
            }
            if (STATES && lane == 0) A.head[job * A.pieces + piece].keep = sum_lost ? __int_as_float(0x7fffffff) : exp2_units(sum);
        } else if (warp == 1) {
            // ---------------- copies ----------------
            const void *mx = &A.map[A.x[job]], *my = &A.map[A.y[job]], *mz = &A.map[A.z[job]];
            const bool sx = J.x.share > 1, sy = J.y.share > 1, sz = J.z.share > 1;
            const uint32_t bytes = (uint32_t)(STATES ? 4 : 6) * A.rows * 128;
            int it = 0;
            for (; it < items; ++it) {
                const int s = it % STAGES;
                if (!wait(sh.info_full[it % INFOS], it / INFOS)) break;
                const Info &I = sh.info[it % INFOS];
                const int t0 = uniform(I.item.t0), h = uniform(I.item.h), hk = uniform(I.item.hk);
                if (it >= STAGES && !wait(sh.empty[s], it / STAGES - 1)) break;
                const uint32_t bar = uniform(smem_u32(&sh.full[s])), to = uniform(sm32 + s * M::STAGE);
                if (elect()) {
                    mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        tma_load_3d(to + M::Y + u * M::ATOM, my, 64 * u, sy ? hk : h, t0, bar);
                        if (!STATES) tma_load_3d(to + M::XT + u * M::ATOM, mx, 64 * u, sx ? hk : h, t0, bar);
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) tma_load_3d(to + M::Z + u * TILE, mz, 64 * u, sz ? hk : h, t0, bar);
                }
                __syncwarp();
                // the next chunk on its way to L2: its copy, once there is room for it, is then a short one
                if (it + 1 < items) {
                    if (!wait(sh.info_full[(it + 1) % INFOS], (it + 1) / INFOS)) break;
                    const Info &F = sh.info[(it + 1) % INFOS];
                    const int t0 = uniform(F.item.t0), h = uniform(F.item.h), hk = uniform(F.item.hk);
                    if (elect()) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            tma_prefetch_3d(my, 64 * u, sy ? hk : h, t0);
                            if (!STATES) tma_prefetch_3d(mx, 64 * u, sx ? hk : h, t0);
                            tma_prefetch_3d(mz, 64 * u, sz ? hk : h, t0);
                        }
                    }
                    __syncwarp();
                }
            }
            // (after a wait that gave up: nothing may be on its way into shared memory when the CTA ends)
            for (int k = max(0, it - STAGES); k < it; ++k)
#pragma unroll 1
                for (uint32_t i = 0; i < kTries && !mbar_try_wait(smem_u32(&sh.full[k % STAGES]), (k / STAGES) & 1); ++i) {}
        } else if (warp == 2) {
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
        } else if (!STATES) {
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
            if (!wait(sh.info_full[it % INFOS], it / INFOS)) break;
            Info &I = sh.info[it % INFOS];
            const int valid = I.item.valid;
            if (keys) {
                if (!wait(sh.full[s], it / STAGES)) break;
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
                            note_first(I.poison, atom * 64 + c0 * 8 + e, reverse ? C - 1 - t : t);
                            I.dirty = 1;
                        }
                    }
                }
                if (it >= SETS && !wait(sh.acc_full[set], it / SETS - 1)) break;      // the operands' last reader
            } else if (zero) {
                if (!wait(sh.full[s], it / STAGES) || (it >= SETS && !wait(sh.acc_full[set], it / SETS - 1))) break;
                if (it == 0)
#pragma unroll 1
                    for (int c = 0; c < 12; ++c)
                        if (c < (FULL ? 12 : 8)) *reinterpret_cast<uint4 *>(row_at + 2 * TILE + (c >> 2) * M::PART + (((i0 >> 3) + (c & 3)) ^ (t & 7)) * 16) = make_uint4(0, 0, 0, 0);
            } else if constexpr (!STATES) {
                uint32_t part[FULL ? 3 : 2][16];
                if (!wait(sh.full[s], it / STAGES) || !wait(sh.pt_full, it)) break;
                tc_fence_after();
                // columns that row t is seen by, in the thread's 32, as bits
                const uint32_t lower = 0xffffffffu >> (31 - lane), mask = t >= valid ? 0u : i0 != 32 * quarter ? 0xffffffffu : reverse ? lower : ~(lower >> 1);
                const float fj = I.fj[t];
                const bool plain = I.plain;
#pragma unroll
                for (int g = 0; g < 32; g += 8) {
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
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = mask >> (g + e) & 1 ? p[e] * __uint_as_float(r[e]) : 0.f;
                    if (dots && i0 == 32 * quarter) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (g + e == lane) {
                                I.own[t] = p[e];
                                p[e] = 0.f;
                            }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        part[0][g / 2 + e] = peel(p[2 * e], p[2 * e + 1]);
                        if (exact) {
                            part[1][g / 2 + e] = peel(p[2 * e], p[2 * e + 1]);
                            if constexpr (FULL) part[2][g / 2 + e] = pack(p[2 * e], p[2 * e + 1]);
                        } else {
                            part[1][g / 2 + e] = pack(p[2 * e], p[2 * e + 1]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.pt_free));
                if (it >= SETS && !wait(sh.acc_full[set], it / SETS - 1)) break;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint8_t *const to = row_at + 2 * TILE + (uint32_t)(((i0 >> 3) + c) ^ (t & 7)) * 16;
#pragma unroll
                    for (int u = 0; u < (FULL ? 3 : 2); ++u) *reinterpret_cast<uint4 *>(to + u * M::PART) = make_uint4(part[u][4 * c], part[u][4 * c + 1], part[u][4 * c + 2], part[u][4 * c + 3]);
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
        const __nv_bfloat16 *const dot_rows = static_cast<const __nv_bfloat16 *>(J.r.p);
        const int dot_heads = dots ? H / J.r.share : 1;
        const uint32_t dot_step = (uint32_t)dot_heads * jb * 2;
        const bool dot_shared = dots && J.r.share > 1;
        const uint32_t row_step = (uint32_t)H * jb * (FULL && !out_bf16 ? 4 : 2);
        float S[COLS];
#pragma unroll
        for (int i = 0; i < COLS; ++i) S[i] = 0.f;
        float *const own_state = A.state + ((size_t)job * A.pieces + piece) * D * D;
        // the state that chunk `it` begins with
        auto enter = [&](const Info &I) {
            const int flags = I.item.flags;
            if (!(flags & (kFromFirst | kFromPiece))) return;
            const int slot = seq_slot(A.c.slot, A.c.num_slots, I.item.n);
            const size_t state = ((size_t)max(slot, 0) * H + I.item.h) * ja * jb;
            // element a of it is at from[a * step]; nothing (zero) without one
            const float *from = flags & kFromFirst ? (first && slot >= 0 && in_b ? first + state + (size_t)b * sb : nullptr)
                                                   : (STATES ? nullptr : own_state - D * D + b);
            int step = flags & kFromFirst ? sa : D;
            if (A.kept && (flags & kOpen)) {
                float *const kept = A.kept + ((size_t)job * A.pieces + piece) * D * D + b;
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
            if (lane == 0) mbar_arrive(smem_u32(&sh.sop_full));
        };
        bool ok = true;
        for (int it = -1; it < items; ++it) {                        // (-1: only the first state goes out)
            const int set = it & (SETS - 1);
            const uint32_t acc = lanes + ACC + set * ACC_STEP;
            Info &I = sh.info[it & (INFOS - 1)];
            int flags = 0, n = 0, h = 0, t0 = 0, valid = 0, chunk = 0;
            bool dirty = false;
            float o[TOKENS];
            if (it >= 0) ok = ok && wait(sh.acc_full[set], it / SETS);
            if (ok && it >= 0) {
                tc_fence_after();
                flags = I.item.flags;
                n = I.item.n;
                h = I.item.h;
                t0 = I.item.t0;
                valid = I.item.valid;
                chunk = I.item.chunk;
                dirty = I.dirty;
                const float keep = I.keep;
                const int poison = dirty ? I.poison[b] : NONE;
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
                if (lane == 0) mbar_arrive(smem_u32(&sh.acc_free[set]));
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
            if (ok) {
                // where the state goes: to an anchor, to the caller, to the piece that goes on
                const int behind = reverse ? chunk * C : chunk * C + valid, begin = t0 - chunk * C;
                const bool at_anchor = anchors && it >= 0 && (reverse ? chunk > 0 && behind % kAnchor == 0 : (flags & kEnds) ? last_anchor : behind % kAnchor == 0);
                const bool to_last = !STATES && (flags & kEnds) && last, to_piece = STATES && it == items - 1;       // (flags of -1: none)
                if (at_anchor || to_last || to_piece) {
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        float *to = nullptr;
                        int step = 0;
                        if (k == 0 && at_anchor) {
                            to = anchors + ((size_t)(anchor_slot(begin, n) + max(0, behind - 1) / kAnchor) * H + h) * ja * jb + b;
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
                // the next chunk's state goes out before this one's rows: the products with it run meanwhile
                if (it + 1 < items) {
                    ok = wait(sh.info_full[(it + 1) % INFOS], (it + 1) / INFOS);
                    if (ok) {
                        enter(sh.info[(it + 1) % INFOS]);
                        if (!STATES) hand_over();
                    }
                }
            }
            if (it < 0) continue;
            if constexpr (STATES) {
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(smem_u32(&sh.info_free[it % INFOS]));
                if (!ok) break;
            } else {
                // a channel a lane, a token a store: 64 bytes of a row a warp
                if (!ok) break;
                const int left = in_b ? valid - TOKENS * part : 0;
                if (FULL && dots) {
                    // the dots of the warp's channels, and the term of the token itself, which is in the rows but not in them
                    const int s = it % STAGES;
                    const char *const r = uniform(reinterpret_cast<const char *>(dot_rows + ((size_t)(t0 + TOKENS * part) * dot_heads + (dot_shared ? I.item.hk : h)) * jb));
                    const uint8_t *const z = sm + s * M::STAGE + M::Z + (b >> 6) * TILE + part * TOKENS * 128 + (b & 7) * 2;
                    float d[TOKENS];
#pragma unroll
                    for (int i = 0; i < TOKENS; ++i) d[i] = load_bf16_if(i < left, r + (2 * b + i * dot_step));
#pragma unroll
                    for (int i = 0; i < TOKENS; ++i) d[i] = i < left ? d[i] * o[i] : 0.f;
#pragma unroll
                    for (int i = 0; i < TOKENS; ++i) {
                        const unsigned short w = *reinterpret_cast<const unsigned short *>(z + i * 128 + (((b >> 3) ^ i) & 7) * 16);
                        o[i] = fmaf(I.own[TOKENS * part + i], __uint_as_float((uint32_t)w << 16), o[i]);
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&sh.info_free[it % INFOS]));        // (an arrival behind the stores would wait for them)
                        mbar_arrive(smem_u32(&sh.empty[s]));
                    }
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
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.info_free[it % INFOS]));
                }
                // (one address for the warp and 32-bit offsets: short code)
                char *const rows = uniform(out + ((size_t)(t0 + TOKENS * part) * H + h) * jb * (FULL && !out_bf16 ? 4 : 2));
                if (FULL && !out_bf16) {
#pragma unroll
                    for (int i = 0; i < TOKENS; ++i) store_if(i < left, rows + (4 * b + i * row_step), o[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < TOKENS; ++i) store_if(i < left, rows + (2 * b + i * row_step), __float2bfloat16_rn(o[i]));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && sh.dead) atomicOr(A.c.status, 2u);
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// The states that pieces leave, one after the other within a pair: S_piece += decay_piece S_before, from the piece that holds the pair's
// start on.  A CTA a slice of the state and first piece.
__global__ void __launch_bounds__(256) join_kernel(const Head *head, float *state, int pieces) {
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

constexpr int MOST_PIECES = 160;

}  // namespace

size_t tc_workspace() { return (size_t)MOST_PIECES * (2 * D * D * sizeof(float) + sizeof(Head)); }

cudaError_t launch_scan_tc(const Call &c, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = smem_attr_once((const void *)tc_kernel<kStates>, (int)kSmem<kStates>, g_attr[0]);
    if (e == cudaSuccess) e = smem_attr_once((const void *)tc_kernel<kPlain>, (int)kSmem<kPlain>, g_attr[1]);
    if (e == cudaSuccess) e = smem_attr_once((const void *)tc_kernel<kFull>, (int)kSmem<kFull>, g_attr[2]);
    if (e != cudaSuccess) return e;
    TcArgs A{};
    A.c = c;
    A.group = 1;
    for (int j = 0; j < c.jobs; ++j)
        for (const Rows *r : {&c.job[j].x, &c.job[j].y, &c.job[j].z})
            if (r->share > A.group) A.group = r->share;
    A.rows = c.T < C ? (c.T < 1 ? 1 : c.T) : C;
    int maps = 0;
    const void *of[4] = {};
    for (int j = 0; j < c.jobs; ++j) {
        const Rows *rows[3] = {&c.job[j].x, &c.job[j].y, &c.job[j].z};
        int *at[3] = {&A.x[j], &A.y[j], &A.z[j]};
        for (int u = 0; u < 3; ++u) {
            int m = 0;
            while (m < maps && of[m] != rows[u]->p) ++m;
            if (m == maps) {
                of[maps++] = rows[u]->p;
                if ((e = make_map(&A.map[m], rows[u]->p, c.T, c.H / rows[u]->share, u == 2 ? c.job[j].b : c.job[j].a, A.rows)) != cudaSuccess) return e;
            }
            *at[u] = m;
        }
    }
    A.pieces = (sms < MOST_PIECES ? sms : MOST_PIECES) / c.jobs;
    A.least = 16;
    A.state = static_cast<float *>(c.pieces);
    A.kept = A.state + (size_t)MOST_PIECES * D * D;
    A.head = reinterpret_cast<Head *>(A.kept + (size_t)MOST_PIECES * D * D);
    if (!c.job[0].first || c.job[0].first != c.job[0].last) A.kept = nullptr;
    // one short sequence: every piece is a whole pair
    const long long longest = c.T / C + 1;
    const bool cut = !(c.N == 1 && longest <= A.least && c.H <= A.pieces);
    if (cut) {
        tc_kernel<kStates><<<A.pieces * c.jobs, THREADS, kSmem<kStates>, s>>>(A);
        count_launch();
        join_kernel<<<dim3(D * D / 1024, A.pieces, c.jobs), 256, 0, s>>>(A.head, A.state, A.pieces);
        count_launch();
    }
    bool plain = true;
    for (int j = 0; j < c.jobs; ++j) plain = plain && c.job[j].out_bf16 && !c.job[j].exact && !c.job[j].dots && !c.job[j].anchors;
    if (plain) tc_kernel<kPlain><<<A.pieces * c.jobs, THREADS, kSmem<kPlain>, s>>>(A);
    else tc_kernel<kFull><<<A.pieces * c.jobs, THREADS, kSmem<kFull>, s>>>(A);
    count_launch();
    return cudaGetLastError();
}

}  // namespace lin
}  // namespace k3kda
