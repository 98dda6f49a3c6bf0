// Host planner. The choices follow the pages' closed forms:
// * wave efficiency (tiles / slots) / ceil(tiles / slots) decides whether a tile shape fills the
//   card ("Kernel development on sm_120", section 4, budget 4; spark-kernels "170 is 2 times 5
//   times 17": a grid that leaves a partial last wave wastes the idle slots for a whole wave);
// * the tile is picked per call: the big tile when its grid fills at least one wave, otherwise
//   a smaller tile, otherwise K is split across the idle slots (spark-kernels, "1024 cubed and the
//   decode shapes" and "170 is 2 times 5 times 17");
// * M <= 64 streams the weights with the skinny kernel, one workgroup per column strip, K split
//   just enough to give the card enough workgroups (spark-kernels, "the decode kernel").
// No autotuning at run time: fixed constants, one closed form per decision ("Kernel development
// on sm_120", section 6, "Autotune").

#include "plan.h"

#include <stdio.h>

#include <algorithm>
#include <cmath>

#include "kernels.h"

namespace glk {

static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

void wave_efficiency(int64_t ctas, int64_t slots, double* eff, int64_t* waves) {
    if (ctas <= 0 || slots <= 0) {
        if (eff) *eff = 0.0;
        if (waves) *waves = 0;
        return;
    }
    const int64_t w = cdiv(ctas, slots);
    if (waves) *waves = w;
    if (eff) *eff = ((double)ctas / (double)slots) / (double)w;
}

bool fast_path_ok(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                  int64_t ldb, const void* C, int64_t ldc) {
    const int64_t kMaxLd = int64_t(1) << 20, kMaxDim = int64_t(1) << 26;
    auto aligned16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    if (!aligned16(A) || !aligned16(B) || !aligned16(C)) return false;
    if ((N & 7) || (K & 7) || (lda & 7) || (ldb & 7) || (ldc & 7)) return false;
    if (lda > kMaxLd || ldb > kMaxLd || ldc > kMaxLd) return false;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return false;
    return true;
}

static void finish_waves(Plan& p) { wave_efficiency(p.grid, p.slots, &p.wave_eff, &p.waves); }

// The split of the strip-major list of (strip, stage) units into `grid` balanced ranges puts
// every range boundary on a strip boundary whenever grid = strips * S: each workgroup then holds
// one piece of one strip, and a strip has exactly S pieces (S = 1: no partials at all), so no
// piece ends mid-range and the fixup is as short as it gets. For each strip width the aligned
// grid takes the most pieces per strip that fit one wave of workgroups; it counts when it
// occupies enough of the CUs: two thirds for up to two 16-row tiles of M, all but a sixteenth
// above that (wider M does more work per byte and wants every CU). The planner takes the largest
// counting grid, and on a tie the one with fewer pieces per strip (less float32 partial traffic).
// 256-column strips are considered only up to two tiles of M: their stages are twice as big, and
// with wider A the ring would be too shallow. Without an aligned grid, Stream-K ranges over one
// workgroup per CU cut 128-column strips wherever they fall.
// The SwiGLU form reads each strip row as two segments, gate and up, of half the strip each:
// there a tie goes to the wider strip instead, which keeps the segments 256 bytes long
// (measured on the 4096 x 22016 gate/up weight at M = 1 and 16: 256-column strips in 2 pieces
// 37.0-37.2 us against 40.2-41.9 us for whole 128-column strips).
static void skinny_layout(int64_t N, int ks, int mtiles, int cus, bool glu, int* strip, int64_t* grid) {
    int best_sw = 0;
    int64_t best_grid = 0, best_s = 0;
    for (int sw : {128, 256}) {
        if (sw == 256 && mtiles > 2) continue;
        const int64_t strips = cdiv(N, sw);
        const int64_t s = std::min<int64_t>(cus / strips, ks);
        if (s < 1) continue;
        const int64_t g = strips * s;
        const bool enough = (mtiles <= 2) ? 3 * g >= 2 * (int64_t)cus : 16 * g >= 15 * (int64_t)cus;
        if (!enough) continue;
        if (g > best_grid || (g == best_grid && (glu ? sw > best_sw : s < best_s))) {
            best_sw = sw;
            best_grid = g;
            best_s = s;
        }
    }
    if (best_sw) {
        *strip = best_sw;
        *grid = best_grid;
    } else {
        *strip = kSkinnyStripMin;
        *grid = std::min<int64_t>(cdiv(N, kSkinnyStripMin) * ks, cus);
    }
}

static Plan plan_skinny(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev, bool glu) {
    Plan p;
    p.kernel = kKernSkinny;
    p.nxcd = dev.nxcd;
    p.mtiles = (int)cdiv(M, 16);
    p.threads = 256;
    p.ks = (int)cdiv(K, kSkinnyStage);
    // one workgroup per CU at most: every launch asks for more than half of a CU's LDS
    p.slots = dev.cus;
    skinny_layout(N, p.ks, p.mtiles, dev.cus, glu, &p.strip, &p.grid);
    p.strips = (int)cdiv(N, p.strip);
    const int64_t units = (int64_t)p.strips * p.ks;
    const int64_t slot_floats = skinny_slot_floats(p.mtiles, p.strip);
    // two partial slots per workgroup; fall back to one unit range per strip (no partials) if
    // the workspace or the counters cannot hold them
    if (2 * p.grid * slot_floats > dev.ws_floats || p.strips > dev.ws_counters) p.grid = p.strips;
    p.ws_floats = 2 * p.grid * slot_floats;
    p.counters = p.strips;
    p.splits = (int)cdiv(p.grid, p.strips);  // pieces per strip, about
    // With 2, 4 or 8 pieces per strip (a divisor of the XCD count) the hardware's round-robin
    // dealing alone gives each XCD the same pieces of many strips: whole rows of one K slice of
    // the weight, where the remap gives it all of K for a few strips, one narrow column block of
    // each row. Measured with one or two 16-row tiles, us: 4096 x 11008 weight 20.8 -> 20.4,
    // 4096 x 4096 12.5 -> 11.0, 8192 x 4096 18.2 -> 16.2, 14336 x 4096 25.4 -> 24.7. Not taken at
    // four tiles (neutral to 2% slower), for the SwiGLU form (1% slower), nor with 16 or 32
    // pieces (1-4% slower).
    if (!glu && p.mtiles <= 2 && p.grid == (int64_t)p.strips * p.splits && p.splits >= 2 &&
        dev.nxcd % p.splits == 0)
        p.nxcd = 1;
    finish_waves(p);
    p.reason = "M <= 64: weights streamed once, " + std::to_string(p.grid) +
               ((p.grid % p.strips == 0) ? " workgroups, each one piece of one strip, over "
                                         : " workgroups over ") +
               std::to_string(units) + " stages of " + std::to_string(p.strip) + "-column strips";
    return p;
}

static void set_tile(Plan& p, int cfg, int64_t M, int64_t N) {
    const TileShape t = tile_shape(cfg);
    p.tile_cfg = cfg;
    p.bm = t.bm;
    p.bn = t.bn;
    p.bk = t.bk;
    p.threads = t.threads;
    p.tiles_m = cdiv(M, t.bm);
    p.tiles_n = cdiv(N, t.bn);
    p.tiles = p.tiles_m * p.tiles_n;
}

static Plan plan_tile(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
    Plan p;
    p.kernel = kKernTile;
    p.nxcd = dev.nxcd;
    // the 256 x 256 tile runs the kernel whose two wave groups alternate MFMA and memory phases:
    // 1.6-2.7% faster than all eight waves in step on every large workload, same bits as far as
    // the tests see (measured interleaved, settled clocks: sq8192 807 against 828 us, mlp_up 300
    // against 309 us, mlp_down 271 against 278 us)
    set_tile(p, kTile256x256pp, M, N);
    // Below one wave of 256x256 tiles, 128x128 tiles: one alone on a CU takes about 60% as long
    // as a 256x256 one (46 against 77 us at K = 4096), and two share a CU (72 KB of LDS and at
    // most 256 registers per lane each), taking about 1.35 times as long together as one alone.
    // So up to two small tiles per CU beat one partial wave of big ones; beyond that the big
    // tiles' lower bytes per flop win (measured, settled clocks: 2048^3 as 256 small tiles 26 us
    // against 41 us as 64 big ones; at K = 4096, 272 to 344 small tiles 61-63 us against 76-77
    // us as 68 to 86 big ones, 512 small tiles 74-76 us against 77 us as 128 big ones, 768
    // small tiles 112 us against 86 us as 192 big ones).
    const int64_t small_tiles = cdiv(M, tile_shape(kTile128x128w4).bm) * cdiv(N, tile_shape(kTile128x128w4).bn);
    if (p.tiles >= dev.cus) {
        p.reason = "256x256 tiles fill at least one wave";
    } else if (small_tiles > 2 * (int64_t)dev.cus) {
        p.reason = "128x128 tiles would need more than two per CU: 256x256 tiles";
    } else {
        set_tile(p, kTile128x128w4, M, N);
        p.reason = small_tiles > dev.cus ? "128x128 tiles, up to two per CU" : "128x128 tiles in one wave";
    }
    if (dev.force_tile_cfg >= 0 && dev.force_tile_cfg < kTileConfigCount) {
        set_tile(p, dev.force_tile_cfg, M, N);
        p.reason = "tile configuration forced";
    }
    const int64_t kt_total = cdiv(K, p.bk);
    p.group_m = (int)std::min<int64_t>(4, p.tiles_m);
    p.sched = kSchedDataParallel;
    p.splits = 1;
    p.kt_per_split = (int)kt_total;
    // workgroups resident at once: one per CU for the 256-wide tile (it takes all of LDS), two for
    // the 128x128 one
    p.slots = (int64_t)dev.cus * (p.tile_cfg == kTile128x128w4 ? 2 : 1);
    // only the smaller tiles carry the split fixup, and only grids of at most one tile per CU
    if (p.tiles <= dev.cus && kt_total > 1 && p.tile_cfg == kTile128x128w4) {
        // split K over the idle CUs; pieces are summed in K order by the last arriver, which
        // reads every other piece's float32 tile (BM*BN*4 bytes), one memory round trip per piece
        // (about 1.2 us), against about 0.4 us per k-step of a lone 128x128 workgroup. So with
        // at most one piece per CU the pieces number about sqrt(kt / 3) (measured, settled
        // clocks: 1024 x 1024 x 8192 in 4 pieces 32 us against 36 us in 8, two per CU; 1024 x
        // 2048 x 4096 in 2 pieces 30 us against 32 us in 4). When more than half the CUs hold a
        // tile, one piece per CU cannot split at all, and two per CU pay: co-resident pieces
        // run together at about 1.35 times a lone one's time, but each costs about 3.5-4 us of
        // fixup, so about sqrt(kt / 8) pieces, and none below 96 k-steps (K = 4096: 144 tiles in
        // 3 pieces 33 us against 46 us, 169 in 3 35.5 against 46, 240 in 2 42 against 46.6, 256
        // (one per CU) in 2 42.4 against 46.2; 256 tiles at K = 11008 in 2 94.9 against 116.2,
        // at K = 3072 35.2 against 36.1, at K = 2048 28.0 against 25.9; 144 tiles at K = 1024 in
        // 3 pieces 19.8 against 15.7 us, 196 at K = 2048 in 2 26.4 against 26.1).
        const int64_t per_cu = dev.cus / p.tiles;
        int64_t s = 1;
        if (per_cu >= 2) {
            int64_t root = 1;
            while ((root + 1) * (root + 1) * 3 <= kt_total) ++root;
            s = std::min<int64_t>(root, per_cu);
        } else if (kt_total >= 96) {
            int64_t root = 1;
            while ((root + 1) * (root + 1) * 8 <= kt_total) ++root;
            s = std::min<int64_t>(root, 2 * dev.cus / p.tiles);
        }
        s = std::max<int64_t>(s, 1);
        const int64_t slot_floats = (int64_t)p.bm * p.bn;
        while (s > 1 && p.tiles * s * slot_floats > dev.ws_floats) --s;
        if (s > 1 && p.tiles > dev.ws_counters) s = 1;
        if (s > 1) {
            p.kt_per_split = (int)cdiv(kt_total, s);
            p.splits = (int)cdiv(kt_total, p.kt_per_split);
            if (p.splits > 1) {
                p.sched = kSchedSplitK;
                p.ws_floats = p.tiles * p.splits * slot_floats;
                p.counters = p.tiles;
                p.reason += ", K split " + std::to_string(p.splits) + " ways";
            }
        }
    }
    p.grid = p.tiles * (p.sched == kSchedSplitK ? p.splits : 1);
    finish_waves(p);
    return p;
}

// A last wave of 256 x 256 tiles that is at most half full takes most of a full wave's time for a
// fraction of its work. Such a product is cut into the largest rectangle of whole tile rows or
// columns that fits in the full waves, planned as before, and the strip left over, planned on its
// own, which must come out as 128 x 128 tiles (at most two per CU, K split over idle CUs). Measured
// against one launch, interleaved, settled clocks, us (last wave's tiles in brackets): 4096 x 4352
// x 4096 (16) 121.7 against 170.5 (hipBLASLt 166.5), 4096 x 4608 x 4096 (32) 134.0 against 172.2,
// 4352^2 x 4096 (33) 136.1 against 172.3, 4096 x 4864 x 4096 (48) 144.1 against 175.7, 4096 x
// 5120 x 4096 (64) 147.1 against 173.3, 4608^3 (68) 181.0 against 194.3, 4096 x 5632 x 4096 (96)
// 168.8 against 178.0, 4096 x 6144 x 4096 (128) 174.3 against 180.1, 6144^3 (64, after two full
// waves) 379.5 against 391.1, 8192 x 8448 x 4096 (32, after four) 428.1 against 458.5; a fuller
// last wave lost (4096 x 11008 x 4096, 176: 284.8 against 278.2; 5120^3, 144: 219.4 against
// 217.2). The SwiGLU form is cut only across rows: its up half sits N weight columns after the
// gate half, so a column strip would need both halves' offsets.
static void cut_sparse_last_wave(Plan& p, int64_t M, int64_t W, int64_t K, const DeviceInfo& dev, bool glu) {
    if (p.kernel != kKernTile || p.tile_cfg != kTile256x256pp || p.sched != kSchedDataParallel) return;
    if (dev.force_tile_cfg >= 0) return;
    const int64_t slots = p.slots;
    const int64_t full = p.tiles / slots, last = p.tiles - full * slots;
    if (full < 1 || last == 0 || 2 * last > slots) return;
    const int64_t room = full * slots;
    int axis = 0;
    int64_t kept = 0, cut = 0;
    if (!glu) {  // keep the first tn tile columns
        const int64_t tn = room / p.tiles_m;
        if (tn >= 1 && tn < p.tiles_n) {
            axis = 1;
            kept = tn * p.tiles_m;
            cut = tn * p.bn;
        }
    }
    {  // keep the first tm tile rows
        const int64_t tm = room / p.tiles_n;
        if (tm >= 1 && tm < p.tiles_m && tm * p.tiles_n > kept) {
            axis = 2;
            kept = tm * p.tiles_n;
            cut = tm * p.bm;
        }
    }
    if (axis == 0) return;
    Plan rest = axis == 1 ? plan_tile(M, W - cut, K, dev) : plan_tile(M - cut, W, K, dev);
    if (rest.tile_cfg != kTile128x128w4) return;
    Plan q = axis == 1 ? plan_tile(M, cut, K, dev) : plan_tile(cut, W, K, dev);
    q.glu = rest.glu = glu;
    q.cut_axis = axis;
    q.cut_at = cut;
    q.ws_floats = std::max(q.ws_floats, rest.ws_floats);
    q.counters = std::max(q.counters, rest.counters);
    q.reason = "a last wave of " + std::to_string(last) + " of " + std::to_string(slots) +
               " 256x256 tiles is cut off: " + q.reason + " over the first " + std::to_string(cut) +
               (axis == 1 ? " columns" : " rows") + ", then the rest: " + rest.reason;
    q.rest.push_back(std::move(rest));
    p = std::move(q);
}

Plan make_plan(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev, bool fast_ok, int force,
               bool glu) {
    Plan p;
    p.glu = glu;
    if (M == 0 || N == 0) {
        p.kernel = kKernNone;
        p.reason = "empty output";
        return p;
    }
    if (K == 0) {
        p.kernel = kKernZero;
        p.grid = 1;
        p.reason = glu ? "K == 0: gate and up are empty sums, silu(0) * 0 = 0" : "K == 0: C is the empty sum";
        return p;
    }
    if (!fast_ok) {
        p.kernel = kKernGeneric;
        p.grid = cdiv(M, 64) * cdiv(N, 64);
        p.threads = 256;
        p.slots = (int64_t)dev.cus * 4;
        finish_waves(p);
        p.reason = "alignment, leading dimension or size outside the fast kernels";
        return p;
    }
    // the fast kernels of the SwiGLU form stream gate and up columns side by side: they are
    // planned over the 2N weight columns
    const int64_t W = glu ? 2 * N : N;
    // the skinny kernel counts its (strip, stage) units in 32 bits
    const bool units_fit = cdiv(W, kSkinnyStripMin) * cdiv(K, kSkinnyStage) <= INT32_MAX;
    const bool skinny = units_fit && ((force == 1) || (force == 0 && M <= 64));
    Plan q = skinny ? plan_skinny(M, W, K, dev, glu) : plan_tile(M, W, K, dev);
    q.glu = glu;
    if (!skinny) cut_sparse_last_wave(q, M, W, K, dev, glu);
    return q;
}

// Block-scaled decode: a workgroup streams the packed weights of 4 column tiles (64 columns) over
// one of S pieces of K, its 4 waves each holding two k-steps of loads in flight in registers.
// Splitting K costs a float32 fixup (about 2 us per call on the 11008 x 4096 weight, measured),
// so K stays whole when one piece per group already covers 60% of the CUs (the 172 groups of an
// 11008-wide weight: 8.3 us at M = 1 against 9.7 at S = 2) and is otherwise cut just far enough to
// cover them all (the 64 groups of a 4096-wide weight: S = 4, 9.7 us, against 14.6 at S = 1 and
// 10.1 at S = 3). Every wave keeps at least one k-step.
// groups of `tpg` column tiles times K pieces over `ks` k-steps (see the comment above)
static Plan decode_groups_plan(int kind, int64_t M, int64_t N, int64_t K, int64_t ks, int tpg,
                               const DeviceInfo& dev) {
    Plan p;
    p.kernel = kind;
    if (M == 0 || N == 0) {
        p.kernel = kKernNone;
        p.reason = "empty output";
        return p;
    }
    if (K == 0) {
        p.kernel = kKernZero;
        p.grid = 1;
        p.reason = "K == 0: C is the empty sum";
        return p;
    }
    // the block-scaled decode's groups go to the XCDs in the hardware's round-robin order: measured
    // against keeping a group's pieces (and neighbouring groups) on one XCD, us, same bits:
    // 4096-wide weight at M = 1, 16, 64 9.75 -> 9.50, 10.27 -> 10.13, 19.21 -> 19.04; 11008-wide
    // at M = 1 7.92 -> 7.62
    p.nxcd = kind == kKernMx ? 1 : dev.nxcd;
    p.threads = 256;
    p.mtiles = (int)cdiv(M, 16);
    p.tiles_n = N / 16;
    p.strips = (int)cdiv(p.tiles_n, tpg);
    p.strip = 16 * tpg;
    p.ks = (int)ks;
    const int64_t per_cu = p.mtiles <= 2 ? 2 : 1;  // waves' registers: two workgroups per CU
    p.slots = per_cu * dev.cus;
    int64_t s = (5 * p.strips >= 3 * (int64_t)dev.cus) ? 1 : cdiv(dev.cus, p.strips);
    s = std::min<int64_t>(s, std::max<int64_t>(1, p.ks / 4));
    const int64_t slot_floats = (int64_t)tpg * p.mtiles * 256;
    while (s > 1 && p.strips * s * slot_floats > dev.ws_floats) --s;
    if (s > 1 && p.strips > dev.ws_counters) s = 1;
    p.splits = (int)s;
    p.grid = p.strips * s;
    p.ws_floats = s > 1 ? p.strips * s * slot_floats : 0;
    p.counters = s > 1 ? p.strips : 0;
    finish_waves(p);
    p.reason = std::string(kind == kKernMx ? "MXFP8 x MXFP4 decode: " : "packed bf16 decode: ") +
               std::to_string(p.strips) + " groups of " + std::to_string(tpg) + " column tiles, K in " +
               std::to_string(s) + " pieces";
    return p;
}

// Workgroups of four column tiles, or of three where that spreads the weight over more CUs: the
// product streams the weight, and a CU left without a workgroup adds nothing to the read rate
// (11008 columns: 172 groups of four against 230 of three, 6% faster at 16 and 64 rows; 4096
// columns: 64 groups of four in 4 K pieces fill 256 CUs exactly and stay).
Plan make_mx_plan(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
    Plan best;
    double best_fill = -1.0;
    for (int tn : {4, 3}) {
        Plan q = decode_groups_plan(kKernMx, M, N, K, K / 128, tn, dev);
        if (q.kernel != kKernMx) return q;
        // how full the rounds of CUs are: the grid over rounds x CUs
        const int64_t rounds = cdiv(q.grid, (int64_t)dev.cus);
        const double fill = (double)q.grid / (double)(rounds * dev.cus);
        if (fill > best_fill + 1e-9) {
            best = q;
            best_fill = fill;
        }
    }
    return best;
}

// The packed bf16 decode reads the same kind of 1 KB operand blocks over 32-k steps.
Plan make_packed_plan(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev) {
    return decode_groups_plan(kKernPacked, M, N, K, K / 32, pk_decode_tiles_per_group(M), dev);
}

// Small outputs leave 128 x 128 tiles on a fraction of the CUs, each copying at the 40-50 bytes a ns
// that one CU takes, and splitting K buys CUs at about 3 us of fixup. 64 x 64 tiles spread the same
// copies over four times as many CUs without it (us, 64 against the best of 128; C = A B^T unless
// noted: 512^3 4.8 against 6.9, 1000^3 8.0 against 11.2, codes 509 x 2501 x 1003 8.2 against 11.7,
// gated forward 300 x 520 x 328 6.0 against 9.0), but copy twice the bytes, which decides once all CUs
// are busy: 2048 x 2048 x 512 10.0 against 8.3, codes 777 x 4096 x 4096 28.3 against 23.1, 2000 x 512 x
// 8192 30.0 against 25.9. So 64 x 64 tiles up to two a CU and 16384 k-steps in all (of 480 random products,
// the bounds of one and a half a CU and 32768 steps lost on 35 where these differ, by 1.16 in the mean:
// codes gated 1404 x 655 x 991, 462 tiles of 16 steps, 7.6 against 12.0; C = A^T B 480 x 2552 x 2306, 320 of
// 73, 21.2 against 16.2), of 32768 where M leaves half of a 128-row tile empty (gated codes 16 x 11008 x
// 4096, 22016 steps: 18.2 of 64 x 64 tiles), and for a quarter as many tiles as CUs whatever K is.
// Pieces of K: a fixup costs like a few k-steps for each piece, so about sqrt(steps / 6) of them (512^3,
// 16 steps: 4.8 us whole, 6.0 in two pieces; codes 300 x 300 x 5008, 79 steps: 9.6 in three, 10.9 in
// two), but none of less than 28 steps once the tiles alone fill the CUs (1000^3, 32 steps: 8.0 whole,
// 9.8 in two), and not a few more workgroups than CUs, whose second round is nearly empty (codes 64
// x 4096 x 11008 in four pieces, 256 workgroups, 15.4; in five, 320 workgroups, 18.8).
Plan make_op_plan(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev, bool glu, bool contiguous) {
    const int64_t tm = cdiv(M, 64), tn = cdiv(glu ? 2 * N : N, 64), kt = cdiv(K, 32);
    const int64_t most = dev.cus + dev.cus / 2;
    const int64_t tiles = 2 * (int64_t)dev.cus, all_steps = tm == 1 ? 32768 : 16384;
    if (tm > tiles || tn > tiles || tm * tn > tiles || (tm * tn * kt > all_steps && tm * tn > dev.cus / 4)) {
        // the gated form is planned over its 2N weight columns: a 256-column tile makes 128 outputs, and
        // the strip of a sparse last wave may be cut off across columns too, as its kernels take the
        // up half's offset apart from the width
        Plan q = make_plan(M, glu ? 2 * N : N, K, dev, true, 2, false);
        // Two pieces on more than two thirds of the CUs, which pay for the other products from 96 k-steps on
        // (make_plan), pay here from 200 where both operands hold the summed index contiguous, whose copies
        // read lines of two k-steps, and from 120 where one is strided. Two pieces against whole, geometric
        // means over 176, 192, 240 and 256 tiles at 96, 120, 141, 170, 200, 256, 344 and 688 k-steps: C = A
        // B^T 1.12, 1.09, 1.15, 1.06, 1.03, 0.95, 1.03, 0.94; codes 1.06, 1.04, 1.08, 1.00, 0.97, 0.93, 0.96,
        // 0.92; C = A^T B 1.01, 0.98, 0.97, 0.94, 0.93, 0.92, 0.90, 0.86; the gated forward 1.01, 0.99, 0.97,
        // 0.93, 0.90, 0.88, 0.86, 0.85 (2048 x 2048 x 11008, us: C = A B^T 90.8 whole and 88.3, C = A^T B 101.7
        // and 98.8; codes 2048 x 2048 x 22016 96.5 and 94.3). A piece takes an even number of k-steps there:
        // one that starts inside a line reads it twice (170 steps, two of 85 against whole: C = A B^T 1.32,
        // codes 1.25).
        if (q.bm == 128 && q.splits == 2 && 3 * q.tiles > 2 * (int64_t)dev.cus) {
            if (kt < (contiguous ? 200 : 120)) {
                q.sched = kSchedDataParallel;
                q.splits = 1;
                q.kt_per_split = (int)kt;
                q.grid = q.tiles;
                q.ws_floats = q.counters = 0;
                q.reason = "128x128 tiles";
                finish_waves(q);
            } else {
                q.kt_per_split += q.kt_per_split & 1;
            }
        }
        q.glu = glu;
        for (Plan& r : q.rest) r.glu = glu;
        if (glu && q.cut_axis == 1) q.cut_at /= 2;
        return q;
    }
    Plan p;
    p.kernel = kKernTile;
    p.glu = glu;
    p.tile_cfg = kTileConfigCount;  // none of make_plan's
    p.bm = p.bn = 64;
    p.bk = 32;
    p.threads = 256;
    p.tiles_m = tm;
    p.tiles_n = tn;
    p.tiles = tm * tn;
    p.nxcd = dev.nxcd;
    p.group_m = (int)std::min<int64_t>(4, tm);
    p.slots = 4 * (int64_t)dev.cus;
    int64_t root = 1;
    while ((root + 1) * (root + 1) * 6 <= kt) ++root;
    int64_t s = std::min<int64_t>(
        {root, std::max<int64_t>(kt / 28, dev.cus / p.tiles), 16, 3 * (int64_t)dev.cus / p.tiles});
    if (p.tiles * s > dev.cus && p.tiles * s <= most) s = dev.cus / p.tiles;
    s = std::max<int64_t>(s, 1);
    while (s > 1 && p.tiles * s * 4096 > dev.ws_floats / 2) --s;  // (two products may share a launch)
    p.kt_per_split = (int)cdiv(kt, s);
    p.splits = (int)cdiv(kt, p.kt_per_split);
    p.sched = p.splits > 1 ? kSchedSplitK : kSchedDataParallel;
    p.grid = p.tiles * p.splits;
    if (p.splits > 1) {
        p.ws_floats = p.grid * 4096;
        p.counters = p.tiles;
    }
    finish_waves(p);
    p.reason = "64x64 tiles";
    return p;
}

// Whether the weight-streaming kernel takes an 8-bit product of at most 64 rows. It has no LDS staging
// to fill and drain, but each of its groups reads all activation rows, where the 64 x 64 tiles read
// them once for 64 weight rows through LDS. Measured with the weights out of the L2s, it wins up to 22
// MB of such reads (us, streaming against tiles: M = 16, 11008 x 4096 12.0 and 12.6; M = 32, 4096 x 4096
// 8.8 and 9.7; M = 64, 1000 x 2000 5.4 and 7.0) and loses beyond (M = 32, 11008 x 4096 14.4 and 12.7; M =
// 64, 4096 x 11008 17.9 and 15.4; gated 11008 x 4096, M = 16 21.7 and 20.6, M = 64 36.8 and 22.2).
bool i8_decode_fits(int64_t M, int64_t K, const Plan& p) {
    return M <= 64 && (int64_t)p.strips * M * K <= int64_t(22) * 1000 * 1000;
}

// The 8-bit product of few rows streams the weight once, and a workgroup of `tn` 16-row tiles also
// reads its K range of all activation rows, which costs like as many weight bytes: the L1 returns
// hits in order behind the stream's misses. So one tile up to 4 rows or while one-tile groups are at
// most two a CU, four tiles beyond (M = 16: 11008 x 4096 weight 12.1 us against 13.9 with one), and
// above 16 rows one, two or four as the weight outgrows the 2 us that summing K pieces costs (M =
// 64: 1000 x 2000 5.3 us with one and 6.3 with two; 2048 x 8192 12.1 with two and 13.4 with four;
// 4096 x 11008 17.9 with four and 20.7 with two). The gated form takes gate and up tiles in pairs, one
// pair up to 16 rows and two for a large weight beyond (M = 64, 11008 x 4096: 37.6 us against 40.1). K is
// split as far as the groups leave CUs idle and 32 k-steps remain to each piece (4 x 2048 x 2048 codes:
// 4.0 us whole, 4.9 in two pieces; 1 x 1000 x 11008: 6.7 in four, 7.0 in three).
Plan make_i8_decode_plan(int64_t M, int64_t N, int64_t K, const DeviceInfo& dev, bool glu) {
    Plan p;
    p.kernel = kKernI8Decode;
    p.glu = glu;
    p.mtiles = (int)cdiv(M, 16);
    const int64_t tiles = cdiv(N, 16), steps = cdiv(K, 64);
    const int64_t weight = (glu ? 2 : 1) * N * K;
    int tn;  // 16-row weight tiles per workgroup
    if (glu)
        tn = p.mtiles > 1 && weight > (int64_t(20) << 20) ? 4 : 2;
    else if (p.mtiles == 1)
        tn = M <= 4 || tiles <= 2 * (int64_t)dev.cus ? 1 : 4;
    else
        tn = weight <= (int64_t(8) << 20) ? 1 : (weight <= (int64_t(20) << 20) ? 2 : 4);
    p.strip = 16 * tn;
    p.strips = (int)cdiv(tiles, glu ? tn / 2 : tn);
    p.ks = (int)steps;
    const int64_t slot_floats = (int64_t)tn * p.mtiles * 256;
    int64_t s = std::max<int64_t>(1, std::min<int64_t>(dev.cus / p.strips, steps / 32));
    while (s > 1 && p.strips * s * slot_floats > dev.ws_floats) --s;
    if (s > 1 && p.strips > dev.ws_counters) s = 1;
    p.splits = (int)s;
    p.grid = p.strips * s;
    p.ws_floats = s > 1 ? p.strips * s * slot_floats : 0;
    p.counters = s > 1 ? p.strips : 0;
    // eight waves where four would leave a CU short of loads in flight: a long K over at most two
    // workgroups a CU (1 x 4096 x 11008: 10.1 us against 10.7), and four tiles of M > 16 (17.9 against 18.6)
    const bool wide = (tn == 1 && p.grid < 2 * (int64_t)dev.cus && steps >= 128) || (!glu && tn == 4 && p.mtiles > 1);
    p.threads = wide ? 512 : 256;
    p.slots = 2 * (int64_t)dev.cus;
    finish_waves(p);
    p.reason = "8-bit decode";  // (short: the call that plans this lasts microseconds)
    return p;
}

// (us of the kernels as they were when a rule was made: both sides of it, on one card.)
// Tiles. Rounds of the tiles that fill the card (one of 256 x 256, two of 128 x 128 or four of 64 x 64 a CU), each at
// what it measured to take for a k-step: 256 x 256 takes 1.68 times a round of 128 x 128 for codes and 1.45 times for bf16,
// 64 x 64 1.1 times. The host knows the number of rows and of groups, and takes a group's last row tile as half full. 128
// x 128 tiles on less than three quarters of the CUs lose to 64 x 64 with more pieces of K, and 256 x 256 ones for
// groups of 100 rows or less to 128 x 128. us, the three sizes in this order: codes 4096 x 4096 x 11008 152, 192, 300; 2048 x
// 4096 x 11008 135, 106, 164; 1024 x 4096 x 4096 52, 33, 38; 1018 rows in 8 groups, 1376 x 512 15.8, 11.0, 10.3; 2048 in 8,
// 4096 x 4096 70.5, 85.7, 102; 2000 in 64, 2048 x 2048 80, 66, 73; bf16 2048 rows in 8 groups, 4096 x 4096 87, 113, 158; 8192 in 64,
// 1376 x 4096 189, 208, 282; 3000 in 32, 2048 x 2048 77, 67, 83.
// Two exceptions: gradients of weights over few rows are a stream of output, which 128 x 128 tiles write faster (16
// rows, 8 groups, 4096 x 1376 25.6, 21.5, 38); and a strided weight is read in rows of a tile's width, 256 bytes of which
// suit a stream for few rows better than 128 where there is one a CU (256 rows in 8 groups, 4096 x 4096 -, 47, 69; 64 in
// 64, 1376 x 4096 -, 83, 90; but 224 tiles, 16 in 8, 4096 x 1376 -, 17.2, 15.7).
// Pieces of K: as many as fill the card where 16 k-steps remain to each, but no more than the square root of a
// quarter of the steps (a sixth for bf16), as a fixup costs like a few steps for each (codes 256 x 4096 x 4096 34 whole, 21
// in four; 128 x 4096 x 4096 20.8 in two, 15.5 in four; 509 x 2501 x 1003 11.0 whole, 11.7 in two). bf16 64 x 64 tiles: one
// workgroup a CU, or two where 20 steps remain (32 where both operands are contiguous); a third on some CUs costs more
// than shorter pieces save (16 rows in 8 groups, 7 with rows, 1376 x 4096, 154 tiles: 25.8 whole, 21.8, 17.8, 19.8,
// 21.4, 21.0 in two to six; 32 in 8, 768 x 8192, 96 tiles: 22.7, 20.8, 22.9 in four to six; 300 in 8, 1376 x 1024, 200
// tiles: 9.0 whole, 10.2 in two; 300 in 3, 1000 x 1000 10.1, 9.3; dA of 128 rows in 4, 1376 x 4096, 256 tiles of 43 steps:
// 11.8, 13.3; of 24 in 4, 2048 x 4096, 64 steps: 15.3, 14.8).
Plan make_group_plan(const GroupShape& g, const DeviceInfo& dev) {
    Plan p;
    p.kernel = kKernTile;
    p.tile_cfg = kTileConfigCount;  // none of make_plan's
    p.bk = 32;
    p.nxcd = dev.nxcd;
    // groups that have rows where every row falls to any of them alike, and the rows of one
    const double miss = g.groups > 1 ? std::pow(1.0 - 1.0 / double(g.groups), double(g.rows)) : 0.0;
    const int64_t parts = std::max<int64_t>(1, std::llround(double(g.groups) * (1.0 - miss)));
    const int64_t each = cdiv(g.rows, parts), cus = dev.cus;
    auto expect = [&](int64_t b) {
        const int64_t rows = g.summed        ? g.groups * cdiv(g.M, b)
                             : g.groups == 0 ? cdiv(g.rows, b)
                                             : std::max(parts, (2 * g.rows / b + parts) / 2);
        return std::max<int64_t>(1, rows * cdiv(g.N, b));
    };
    const int64_t high = g.summed ? g.M : each, kt = cdiv(g.summed ? each : g.K, 32);
    // Few 256 x 256 tiles past whole rounds are in pieces of K: up to the square root of an eighth of the k-steps (a quarter
    // for codes), from 48 steps. The grid of a grouped product has a workgroup for each slot of the workspace. us whole
    // and in 2, 4 and 8 pieces, 16 tiles past a round: codes 4096 x 4352 x 11008 251, 212, 187, 188; x 4096 101, 94, 85, 94; x 2048 58, 60, 56, 67;
    // bf16 436, 354, 314, 303; 169, 145, 132, 135; 91, 83, 79, 87; x 1024 52, 52, 53, 64.
    const int64_t slots = g.summed || kt < 48 ? 0 : dev.ws_floats / (256 * 256);
    while (slots > 1 && p.tail < 8 && (p.tail + 1) * (p.tail + 1) * (g.pairs ? 4 : 8) <= kt) ++p.tail;
    int64_t rounds256 = cdiv(expect(256), cus) * 100, extra = slots;  // hundredths; workgroups
    if (g.groups == 0 && !g.summed) {  // (the tiles are known)
        const int64_t rest = expect(256) % cus, pieces = rest ? std::min<int64_t>({slots / rest, cus / rest, p.tail}) : 1;
        if (pieces > 2) rounds256 -= 50 - 100 / pieces;  // (the sum takes about half a round)
        if (pieces < 2) p.tail = 1;
        extra = rest * (pieces - 1);
    }
    const int64_t t256 = rounds256 * (g.pairs ? 168 : 145) / 100, t128 = cdiv(expect(128), 2 * cus) * 100,
                  t64 = cdiv(expect(64), 4 * cus) * 110;
    int bm = t128 < t64 && 4 * expect(128) >= 3 * cus && high > 16 && g.N > 64 ? 128 : 64;
    if (high > 100 && g.N > 100 && 2 * expect(256) >= cus && t256 < std::min(t128, t64) && !(g.summed && each <= 64)) bm = 256;
    if (g.strided && each <= 32 && expect(128) >= cus) bm = 128;
    if (g.tile) bm = g.tile;
    // a launch holds 2^32 - 1 threads
    auto fits = [&](int64_t b) {
        const int64_t rows = g.summed ? g.groups * cdiv(g.M, b) : most_row_tiles(g.rows, g.groups, b);
        return rows <= kMostThreads / (b == 256 ? 512 : 256) / cdiv(g.N, b);
    };
    while (bm < 256 && !fits(bm)) bm *= 2;
    p.bm = p.bn = bm;
    p.threads = bm == 256 ? 512 : 256;
    p.tiles_n = cdiv(g.N, bm);
    p.tiles_m = g.summed ? cdiv(g.M, bm) : most_row_tiles(g.rows, g.groups, bm);
    p.tiles = (g.summed ? g.groups : 1) * p.tiles_m * p.tiles_n;
    p.group_m = (int)std::min<int64_t>(4, p.tiles_m);
    int64_t s = 1;
    if (bm < 256) {
        const int64_t tiles = expect(bm);
        if (bm == 64 && !g.pairs && !g.summed) {
            s = std::max(std::min(cus / tiles, kt / 16), std::min(2 * cus / tiles, kt / (g.strided ? 20 : 32)));
        } else {
            s = std::min((g.pairs ? 4 : 3) * cus / (bm == 128 ? 2 : 1) / tiles, kt / 16);
        }
        int64_t root = 1;
        while ((root + 1) * (root + 1) * (g.pairs ? 4 : 6) <= kt) ++root;
        s = std::max<int64_t>(1, std::min<int64_t>({s, root, 16}));
        // (both gradients may share a launch)
        while (s > 1 && p.tiles * s * bm * bm > dev.ws_floats / (g.pairs || g.strided ? 1 : 2)) --s;
        if (s > 1 && p.tiles > dev.ws_counters / 2) s = 1;
    }
    int64_t per = std::max<int64_t>(1, cdiv(kt, s));
    if (g.pairs) per += per & 1;
    p.kt_per_split = (int)per;
    p.splits = (int)(g.summed ? s : std::max<int64_t>(1, cdiv(kt, per)));
    p.sched = p.splits > 1 ? kSchedSplitK : kSchedDataParallel;
    p.slots = (bm == 256 ? 1 : bm == 128 ? 2 : 4) * cus;
    p.grid = p.tiles * p.splits;
    if (p.splits > 1) {
        p.ws_floats = p.grid * bm * bm;
        p.counters = p.tiles;
    }
    if (bm != 256) p.tail = 1;
    if (p.tail > 1) {
        p.grid += extra;
        p.ws_floats = slots * 256 * 256;
        p.counters = slots;
    }
    finish_waves(p);
    p.reason = "grouped rows";
    return p;
}

// The 8-bit floating-point product of few rows streams the weight once for each row tile, and as in the integer
// form a workgroup's activations cost like as many weight bytes. us a call, weights from HBM:
// * tn: one weight tile up to two a CU (8 x 4096 x 4096 7.6, 8.7 with two), then four (16 x 11008 x 4096 14.7 and 15.4
//   with one); up to 4 rows a group one (1 x 11008 x 4096 11.9, 13.3 with two) until there are eight a CU, then two (41
//   of 64 groups of 1376 x 4096: 46.4, 48.6 with one, 50.8 with four). Above 16 rows one, two or four as the weight
//   outgrows the sum of K pieces (64 x 1000 x 2000 7.6, 8.5 with two, 11.2 with four; 48 x 2048 x 8192 12.7 with two, 14.2 with
//   one, 17.4 with four; 64 x 11008 x 4096 24.6 with four and 29.7 with two).
// * pieces: as far as the strips leave CUs idle and 10 blocks of 128 remain to each, 4 above 16 rows (16 x 1000 x 4096,
//   32 blocks: 6.5 in two, 6.3 in three; 4 x 2048 x 2048, 16 blocks: 4.7 whole, 5.5 in two; 64 x 1000 x 2000, 16: 8.2 whole,
//   7.6 in four). More than one workgroup a CU costs more than the CUs that it fills (172 strips: 64 x 11008 x 4096 24.6 whole,
//   34.5 in two, 38.3 in three; 32 x 11008 x 4096 17.1, 20.0, 21.3; 16 x 11008 x 4096 14.7, 17.3, 18.4).
// Four waves: eight were 0.4 to 3 us slower, or at best 3% faster.
Plan make_f8_decode_plan(int64_t rows, int64_t N, int64_t K, int64_t groups, const DeviceInfo& dev) {
    Plan p;
    p.kernel = kKernF8Decode;
    // The row tiles of one strip and piece, neighbours in the order of units, go to one XCD and share its L2: a group of more
    // than 16 rows reads its weight once for each XCD else (us with and without: 128 rows all of one of 8 groups, 4096 x
    // 4096 25.2 and 27.3, of two 29.8 and 32.2; 64 of two 24.8 and 26.1; 64 in 41 of 64, 1376 x 4096 46.2 and 46.2). A plain
    // product is one row tile (1 x 11008 x 4096 10.6 and 10.5).
    p.nxcd = groups > 0 ? dev.nxcd : 1;
    const int64_t parts = std::max<int64_t>(1, std::min(groups, rows));  // that can have rows
    const int64_t each = cdiv(rows, parts);
    p.mtiles = each <= 16 ? 1 : each <= 32 ? 2 : 4;
    const int64_t row_tiles = parts * cdiv(each, 16 * p.mtiles);  // as an even router would make them
    const int64_t tiles = cdiv(N, 16) * row_tiles, steps = cdiv(K, 128), cus = dev.cus;
    const int64_t weight = N * K * parts;
    int tn;  // 16-row weight tiles per workgroup
    if (p.mtiles > 1)
        tn = weight <= (int64_t(8) << 20) ? 1 : (weight <= (int64_t(20) << 20) ? 2 : 4);
    else if (each <= 4)
        tn = tiles >= 8 * cus ? 2 : 1;
    else
        tn = tiles <= 2 * cus ? 1 : 4;
    p.strip = 16 * tn;
    p.strips = (int)cdiv(cdiv(N, 16), tn);
    p.ks = (int)steps;
    const int64_t all = p.strips * most_row_tiles(rows, groups, 16 * p.mtiles);
    const int64_t slot_floats = (int64_t)tn * p.mtiles * 256;
    int64_t s = std::max<int64_t>(1, std::min<int64_t>(cus / (p.strips * row_tiles), steps / (p.mtiles == 1 ? 10 : 4)));
    while (s > 1 && all * s * slot_floats > dev.ws_floats) --s;
    if (s > 1 && all > dev.ws_counters) s = 1;
    p.splits = (int)s;
    p.grid = all * s;
    p.ws_floats = s > 1 ? all * s * slot_floats : 0;
    p.counters = s > 1 ? all : 0;
    p.threads = 256;
    p.slots = 2 * cus;
    finish_waves(p);
    p.reason = "8-bit float decode";
    return p;
}

// Whether the weight-streaming kernel is made for the product: a plain one of at most 64 rows (us, streaming against
// tiles: 64 x 11008 x 4096 24.6 and 35.3, 64 x 4096 x 11008 24.0 and 28.1, 64 x 512 x 1024 6.5 and 8.6), a grouped one of
// at most 16 rows a group in the mean.
bool f8_decode_fits(int64_t rows, int64_t groups) { return groups == 0 ? rows <= 64 : rows <= 16 * groups; }

// Whether it takes the product from the tiles. The host knows the rows a group in the mean and not how a router deals them,
// and the kernel reads the weight of a group once for every 16 of its rows, the tiles once for every 64. us, streaming against tiles,
// rows over nearly all groups, over a quarter of them and all in one: 64 groups, 4096 to 1376, 1 row a group 46 and 56, 22
// and 22, 12 and 19; 2 62 and 81, 23 and 22, 18 and 20; 4 64 and 89, 32 and 23, 24 and 21; 8 78 and 85, 46 and 24, 38 and 23; 16 98 and 97, 75
// and 27, 69 and 26. 8 groups, 4096 x 4096, 4 a group 26 and 25, 15 and 16, 12 and 15; 8 26 and 25, 25 and 16, 16 and 15; 16 34 and 26, 30 and 17, 25
// and 16.
bool f8_decode_pays(int64_t rows, int64_t groups) { return f8_decode_fits(rows, groups) && (groups == 0 || rows <= 4 * groups); }

static const char* kernel_name(int k) {
    switch (k) {
        case kKernNone: return "none";
        case kKernZero: return "zero";
        case kKernGeneric: return "generic";
        case kKernTile: return "tile";
        case kKernSkinny: return "skinny";
        case kKernMx: return "mx";
        case kKernPacked: return "packed";
        case kKernI8Decode: return "i8_decode";
        case kKernF8Decode: return "f8_decode";
        default: return "?";
    }
}

std::string plan_json(const Plan& p, int64_t M, int64_t N, int64_t K) {
    char buf[4096];
    snprintf(buf, sizeof buf,
             "{\"M\": %lld, \"N\": %lld, \"K\": %lld, \"kernel\": \"%s\", \"bm\": %d, \"bn\": %d, "
             "\"bk\": %d, \"threads\": %d, \"tiles_m\": %lld, \"tiles_n\": %lld, \"tiles\": %lld, "
             "\"schedule\": \"%s\", \"splits\": %d, \"kt_per_split\": %d, \"group_m\": %d, "
             "\"nxcd\": %d, \"mtiles\": %d, \"strip\": %d, \"strips\": %d, \"ks\": %d, \"grid\": %lld, "
             "\"slots\": %lld, \"waves\": %lld, \"wave_eff\": %.6f, \"ws_floats\": %lld, "
             "\"op\": \"%s\", \"reason\": \"%s\"}",
             (long long)M, (long long)N, (long long)K, kernel_name(p.kernel), p.bm, p.bn, p.bk,
             p.threads, (long long)p.tiles_m, (long long)p.tiles_n, (long long)p.tiles,
             p.kernel == kKernTile ? (p.sched == kSchedSplitK ? "split-k" : "data-parallel")
                                   : (p.kernel == kKernSkinny || p.kernel == kKernMx || p.kernel == kKernPacked ||
                                           p.kernel == kKernI8Decode || p.kernel == kKernF8Decode
                                          ? "strips"
                                          : "-"),
             p.splits, p.kt_per_split, p.group_m, p.nxcd, p.mtiles, p.strip, p.strips, p.ks,
             (long long)p.grid, (long long)p.slots, (long long)p.waves, p.wave_eff,
             (long long)p.ws_floats,
             p.kernel == kKernMx ? "mx" : (p.kernel == kKernPacked ? "packed" : (p.glu ? "swiglu" : "gemm")),
             p.reason.c_str());
    std::string s(buf);
    if (p.cut_axis != 0 && !p.rest.empty()) {
        // the strip left over: its own plan, over its own sizes
        const int64_t Mr = p.cut_axis == 2 ? M - p.cut_at : M;
        const int64_t Nr = p.cut_axis == 1 ? N - p.cut_at : N;
        s.pop_back();
        s += ", \"cut\": {\"axis\": \"" + std::string(p.cut_axis == 1 ? "n" : "m") +
             "\", \"at\": " + std::to_string(p.cut_at) + ", \"rest\": " + plan_json(p.rest[0], Mr, Nr, K) + "}}";
    }
    return s;
}

}  // namespace glk
