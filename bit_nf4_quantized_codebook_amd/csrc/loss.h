// Softmax cross entropy of the output head: what its kernels share (gfx950).
//
// Tokens without a label take no part: the others' indices are gathered once ("live rows", in
// order), every kernel counts in live rows, and how many there are stays on the device.
//
// Logits are handled in units of log2: l = z log2(e), and a row's reference c is an integer, so that
// moving a sum or a probability from one reference to another is a product with a power of two,
// which rounds nothing.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4k {

constexpr int LT = 256;                  // tokens, vocabulary rows or columns of dX of a tile
constexpr int LSTEP = 64;                // reduction of one step of a tile's loop
constexpr int64_t LBLOCK = LT * LSTEP;   // elements of one step's operand tile (32 KB)
constexpr int kLossJoinRows = 8;         // rows of a workgroup that joins the tiles
constexpr int kLossJoinRowsNarrow = 2;   // the same for few tokens
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;

// Per-row state in the workspace; row arrays have Mp = M rounded up to 256 entries.
struct LossRows {
    int32_t *count;        // [2] live rows; workgroups of a join that have ended (few tokens, forward)
    double *sums;          // [a join's workgroups] sums of the losses of each workgroup of the last join
    int32_t *row;          // [M] live row -> token
    int32_t *label;        // [M] its label; -1: out of the vocabulary (its results are NaN)
    float *zl;             // [M] the label's logit in log2 units (unset without one)
    float *S;              // [M] sum over the other vocabulary rows of 2^(l - c)
    float *a, *b;          // [M] dX = b (a sum P W - W[label]); a: between pieces, the sum of P
};

// Tiles of rows and columns, numbered along the columns within groups of four tiles of rows (an XCD's concurrent
// tiles then share both operands in its L2).
__host__ __device__ __forceinline__ void loss_place(int ntm, int ntn, int t, int &tm, int &tn) {
    const int grp = t / (4 * ntn), first = 4 * grp, size = ntm - first < 4 ? ntm - first : 4, in = t - 4 * grp * ntn;
    tm = first + in % size;
    tn = in / size;
}

// How dX's product shares its tiles' reductions of `steps` steps among 256 workgroups: whole rounds of tiles first, a
// tile a workgroup.  The `rest` tiles are split ks ways, len steps each.  Where that leaves workgroups over (extra), the
// ks parts are cut to about rest steps / 256 and the tails they leave, laid end to end, go to the extra ones in equal
// runs.  A split tile's parts are float32 partials.  (All of it laid end to end in 256 runs had as many partials and
// every workgroup at another step: nothing to share in the L2s, 527 instead of 414 us for 112 tiles of 500 steps.)
// The extra ones are used where the time they save, at 1.6 us a step, exceeds their partials', 0.114 us each to write
// and read.
struct LossShares {
    int tiles, steps, whole, rest, ks, len, extra, tail;
    __host__ __device__ LossShares(int tiles_, int steps_) : tiles(tiles_), steps(steps_) {
        whole = tiles / 256 * 256;
        rest = tiles - whole;
        ks = extra = tail = 0;
        len = steps;
        if (!rest) return;
        ks = 256 / rest;
        if (ks > steps / 8) ks = steps / 8 > 0 ? steps / 8 : 1;
        len = (steps + ks - 1) / ks;
        ks = (steps + len - 1) / len;
        // (starting and storing a part takes about six steps' time, once more for every tile of a run)
        const int cut = (int)((int64_t)rest * (steps + 6) / 256), over = 256 - rest * ks;
        // in units of 1/1000 us; a run of tails may begin in one tile and end in another
        const int64_t shorter = (int64_t)(len - cut) * 1600, parts = (int64_t)(over + rest + (ks == 1 ? rest : 0)) * 114;
        if (over <= 0 || cut < 8 || ks * cut >= steps || shorter <= parts) return;
        len = cut;
        extra = over;
        tail = steps - ks * len;
    }
    __host__ __device__ __forceinline__ bool partial() const { return ks > 1 || extra; }
    // runs of the tails, in steps of all tails
    __host__ __device__ __forceinline__ int64_t begin(int e) const { return (int64_t)rest * tail * e / extra; }
    __host__ __device__ __forceinline__ int run_of(int64_t u) const {
        const int64_t all = (int64_t)rest * tail;
        return (int)(((u + 1) * extra + all - 1) / all) - 1;
    }
    // partials: part j of tile x; a run's part in the tile that it begins in; a tile whose tail begins inside a run
    __host__ __device__ __forceinline__ int slot_part(int j, int x) const { return j * rest + x; }
    __host__ __device__ __forceinline__ int slot_run(int e, int x) const {
        return ks * rest + (begin(e) >= (int64_t)x * tail ? e : extra + x);
    }
};

// Tiles of the logits of a piece, for ntm tiles of rows and ntn of the vocabulary.  Where they fill the chip's last round
// at most half, that round's tiles are cut in two along the vocabulary (777 x 50001 x 8192 with about 700
// labelled 1183 us, 1219 uncut): their second halves' statistics stand ntn entries further in the tables.
//
// The last tile of rows is a whole one however few of them are live.  Tiles of 128 tokens there took 923 us against 796 at
// 1639 x 32000 x 4096 (a step of half the MFMAs does not hide its loads with two stages), and 128 x 512 ones 1343 against
// 1335 at 777 x 50001 x 8192, all labelled (both with the gradient): rows of zeros cost the MFMAs little power, and the wide
// tiles read W once more.
struct LossTiles {
    int ntm, ntn, whole;      // whole: tiles that are not cut, the first ones
    __host__ __device__ LossTiles(int m, int n) : ntm(m), ntn(n) {
        const int64_t t = (int64_t)m * n;
        const int rest = (int)(t % 256);
        whole = (int)(rest <= 128 ? t - rest : t);
    }
    __device__ __forceinline__ void place(int t, int &tm, int &tn) const { loss_place(ntm, ntn, t, tm, tn); }
    // the first tile of the vocabulary that is cut for these rows; all after it are too
    __device__ __forceinline__ int first_cut(int tm) const {
        const int first = tm & ~3, size = ntm - first < 4 ? ntm - first : 4, left = whole - first * ntn - (tm - first);
        return left <= 0 ? 0 : min((left + size - 1) / size, ntn);
    }
};

struct LogitsArgs {
    const uint16_t *W, *X;
    int64_t V, K;
    LossRows r;
    int32_t Mp;
    int32_t tile0, ntile;     // vocabulary tiles of this piece
    const float *ref;         // [M] references, or NULL: 0
    float *tref, *tsum;       // [2 ntile][Mp]: a tile's reference and its sum of 2^(l - reference)
    float *tp;                // the same of P, which is rounded, or NULL
    uint16_t *P;              // 2^(l - reference) in bf16, or NULL; blocks of one step (see loss_logits.hip)
    int32_t psteps;           // steps of P's row of blocks
};
hipError_t launch_loss_logits(const LogitsArgs &a, hipStream_t stream);

// dX's product over a piece.  Where a tile's reduction is not shared, the product itself adds what earlier pieces
// left (sum32, moved from the references c_old to c) and writes sum32 or, with the last piece, dX.
struct LossDxArgs {
    const uint16_t *P, *W;
    int64_t V, K, v0;         // v0: first vocabulary row of the piece
    LossRows r;
    int32_t Mp, steps;
    float *part;              // [256 + rest] blocks of 256 x 256 float32 (row: token)
    float *sum32;             // [Mp, K]; NULL: one piece only
    const float *c, *c_old;   // c_old NULL: the first piece
    uint16_t *dX;             // NULL: not the last piece
    int64_t M;
    float *mean;              // written by the fold, or NULL
};
hipError_t launch_loss_dx(const LossDxArgs &a, hipStream_t stream);
// the same for the tiles with partials
hipError_t launch_loss_fold(const LossDxArgs &a, hipStream_t stream);

// labels -> live rows; loss and dX of the other tokens set to zero
hipError_t launch_loss_prep(const int64_t *labels, int64_t M, int64_t V, int64_t K, const LossRows &r, float *loss,
                            uint16_t *dX, hipStream_t stream);
// the tiles' references and sums into the rows' (c_in NULL: the first), and P's tiles brought from their own references to
// the rows' where any differs
struct LossJoin {
    LossRows r;
    int64_t M;
    int32_t Mp;
    const float *tref, *tsum, *tp;
    int32_t ntile;
    const float *c_in;
    float *c_out;
    uint16_t *P;              // or NULL: the forward
    int32_t prows;            // rows of one of P's blocks
    // the last join: losses, the sums for their mean, and with grad the coefficients of dX
    bool last, grad;
    const float *dloss;
    float *loss, *mean;
    bool tickets;             // its last workgroup writes the mean (count[1] is 0 before)
};
// narrow: the tables of loss_narrow.hip
hipError_t launch_loss_join(const LossJoin &a, bool narrow, hipStream_t stream);
// the mean from the last join's sums (with grad, dX's last launch writes it; one workgroup of the join writes it itself, and
// with tickets the join does)
hipError_t launch_loss_mean(const LossRows &r, int64_t M, float *mean, hipStream_t stream);

// by 256 threads
__device__ __forceinline__ void loss_write_mean(const double *sums, int n, int count, float *mean) {
    __shared__ double total[256];
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += 256) s += sums[i];
    total[threadIdx.x] = s;
    __syncthreads();
    for (int d = 128; d > 0; d >>= 1) {
        if ((int)threadIdx.x < d) total[threadIdx.x] += total[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) mean[0] = count ? (float)(total[0] / count) : 0.0f;
}

// Up to kLossNarrowMaxM tokens, in one piece; up to kLossNarrowMaxM2 where the vocabulary is at most kLossNarrowMaxTiles
// tiles of 256, half a round of the chip (with the gradient, 200 tokens: 32000 x 4096 183 us, tiles of 256 189, of those
// 60 labelled 120 and 156; 8000 x 4096 85 and 107; 160 x 4000 x 1024 42 and 59.  Above: 32769 x 4096 250 and 210, of 200
// labelled 60 143 and 182; 50001 x 4096 298 and 263, 120 labelled 247 and 241, 60 203 and 225: few labels would want the narrow
// tiles there too, but how many there are is known on the device only).
constexpr int64_t kLossNarrowMaxM = 128, kLossNarrowMaxM2 = 256, kLossNarrowMaxTiles = 128;
struct LossNarrowPlan {
    int32_t MT;               // tokens there may be: 64, 128 or 256
    int32_t steps, per;       // steps of 64 vocabulary rows: all, and of dX's workgroup
    int32_t splits;           // dX's workgroups along the vocabulary
    size_t parts;             // float32 partials
};
LossNarrowPlan loss_narrow_plan(int64_t M, int64_t V, int64_t K);
struct LossNarrow {
    const uint16_t *W, *X;
    int64_t V, K, M;
    const int64_t *labels;
    LossRows r;
    LossNarrowPlan n;
    float *tref, *tsum, *tp;  // [M][steps]; tp: as in LogitsArgs
    uint16_t *P;              // [steps] blocks of MT rows; NULL: the forward
    float *part;
    float *loss, *mean;
    uint16_t *dX;
};
hipError_t launch_loss_narrow_logits(const LossNarrow &g, hipStream_t stream);
hipError_t launch_loss_narrow_dx(const LossNarrow &g, hipStream_t stream);        // with dX and the mean

// the forward for up to kLossGemvMaxM tokens
constexpr int64_t kLossGemvMaxM = 16;
struct LossGemv {
    const uint16_t *W, *X;
    int64_t V, K, M;
    const int64_t *labels;
    float2 *table;            // [M][ceil(V / 16)] reference and sum of each 16 vocabulary rows
    float *zl, *each;         // [M]
    int32_t *done;
    float *loss, *mean;
};
hipError_t launch_loss_gemv(const LossGemv &g, hipStream_t stream);

}  // namespace nf4k
