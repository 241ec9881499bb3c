// How dX's product of the loss shares its tiles' reductions (LossShares), on the host: over many numbers of tiles and steps,
// every step of every tile is taken once, every partial is written once and inside the buffer, and the fold of a tile reads
// exactly its own, in the order of their steps.  Prints what it saw.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "loss.h"

using nf4k::LossShares;

static void need(bool ok, int tiles, int steps, const char *what) {
    if (ok) return;
    std::printf("tiles %d steps %d: %s\n", tiles, steps, what);
    std::exit(1);
}

struct Partial {
    int tile = -1, from = 0, to = 0;
};

static int with_runs = 0, crossing = 0, split = 0;

static void check(int tiles, int steps) {
    const LossShares sh(tiles, steps);
    need(sh.whole % 256 == 0 && sh.whole + sh.rest == tiles && sh.rest < 256, tiles, steps, "tiles");
    if (!sh.rest) return;
    // as loss_dx_kernel's workgroups take them: XCD i of 8 parts i/8 .. (i+1)/8, its 32 workgroups one each, those left over a
    // run each
    std::vector<Partial> slots(256 + sh.rest);
    std::vector<std::vector<int>> taken(sh.rest, std::vector<int>(steps, 0));
    std::vector<int> part_by(sh.ks * sh.rest, 0), run_by(sh.extra, 0);
    auto take = [&](int x, int from, int to, int slot) {
        need(x >= 0 && x < sh.rest && from < to && from >= 0 && to <= steps, tiles, steps, "a share out of range");
        for (int k = from; k < to; ++k) ++taken[x][k];
        if (!sh.partial()) return;
        need(slot >= 0 && slot < (int)slots.size() && slots[slot].tile < 0, tiles, steps, "a slot written twice or out of range");
        slots[slot] = Partial{x, from, to};
    };
    const int parts = sh.ks * sh.rest;
    for (int block = 0; block < 256; ++block) {
        const int xcd = block & 7, slot = block >> 3, p0 = parts * xcd / 8, p1 = parts * (xcd + 1) / 8, mine = p0 + slot;
        if (mine < p1) {
            ++part_by[mine];
            const int j = mine / sh.rest, x = mine % sh.rest, kb = j * sh.len;
            take(x, kb, kb + (sh.len < steps - kb ? sh.len : steps - kb), sh.slot_part(j, x));
        } else if (sh.extra) {
            const int run = 32 * xcd - p0 + slot - (p1 - p0);
            need(run >= 0 && run < sh.extra, tiles, steps, "a run out of range");
            ++run_by[run];
            int tiles_of = 0;
            for (int64_t at = sh.begin(run), until = sh.begin(run + 1); at < until; ++tiles_of) {
                const int x = (int)(at / sh.tail), in = (int)(at - (int64_t)x * sh.tail);
                const int n = (int)(until - at < sh.tail - in ? until - at : sh.tail - in);
                take(x, sh.ks * sh.len + in, sh.ks * sh.len + in + n, sh.slot_run(run, x));
                at += n;
            }
            need(tiles_of > 0, tiles, steps, "an empty run");
            crossing += tiles_of > 1;
        }
    }
    for (int n : part_by) need(n == 1, tiles, steps, "a part not taken once");
    for (int n : run_by) need(n == 1, tiles, steps, "a run not taken once");
    for (const auto &t : taken)
        for (int n : t) need(n == 1, tiles, steps, "a step not taken once");
    with_runs += sh.extra > 0;
    split += sh.partial();
    if (!sh.partial()) return;
    size_t read = 0, written = 0;
    for (const Partial &p : slots) written += p.tile >= 0;
    for (int x = 0; x < sh.rest; ++x) {
        // as loss_fold_kernel reads them
        const int e0 = sh.extra ? sh.run_of((int64_t)x * sh.tail) : 0;
        const int n = sh.ks + (sh.extra ? sh.run_of((int64_t)(x + 1) * sh.tail - 1) - e0 + 1 : 0);
        int at = 0;
        for (int i = 0; i < n; ++i, ++read) {
            const Partial &p = slots[i < sh.ks ? sh.slot_part(i, x) : sh.slot_run(e0 + i - sh.ks, x)];
            need(p.tile == x && p.from == at, tiles, steps, "the fold reads another tile's partial, or out of order");
            at = p.to;
        }
        need(at == steps, tiles, steps, "the fold misses steps");
    }
    need(read == written, tiles, steps, "partials that no fold reads");
}

int main() {
    for (int rest = 1; rest < 256; ++rest)
        for (int steps = 4; steps <= 520; steps += 4) check(rest, steps);      // four a tile of the vocabulary
    for (int rest = 1; rest < 256; rest += 5)
        for (int steps = 524; steps <= 16384; steps += 4 * 97) check(rest + 256 * (steps % 3), steps);
    check(256, 500);
    check(512, 4);
    std::printf("split %d, with runs %d, runs over two tiles %d\n", split, with_runs, crossing);
    return with_runs > 1000 && crossing > 1000 ? 0 : 1;
}
