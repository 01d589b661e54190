// The attention kernels' deal of tiles to workgroups, on the host: for each
// line "held passing group offset causal by_keys heads" of the input, every
// workgroup's walk; prints "ok grid shared" or what is wrong.
#include <stdio.h>
#include <string.h>

#include <vector>

#include "svdq_layout.h"

using namespace svdq;

int main() {
  long long held, passing, group, offset, causal, by_keys, heads;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld", &held, &passing, &group, &offset, &causal, &by_keys, &heads) == 7) {
    const AttnCost c = {(int)held, (int)passing, (int)group, (int)offset, (int)causal, (int)by_keys};
    const AttnPlan p = attn_plan(c, heads);
    const int units = p.blocks * (int)heads;
    std::vector<std::vector<AttnPiece>> of(units);
    std::vector<std::vector<int>> by(units);
    const char* bad = nullptr;
    std::vector<int> slots(2 * p.grid, 0), seen(p.grid, 0), w0(units, -1), w1(units, -1);
    AttnShares shares;
    if (p.shared) attn_shares(c, p, &shares);
    int most = 0, least = 1 << 30;
    for (int id = 0; id < p.grid && !bad; ++id) {
      const int w = attn_place(p, id);
      if (w < 0 || w >= p.grid || seen[w]++) { bad = "two workgroups at one place"; break; }
      AttnWalk walk(p, w, p.shared ? shares.at[w] : AttnStart{0, 0, 0});
      AttnWhole whole;
      AttnPiece o;
      int n = 0;
      while (p.shared ? walk.next(c, p, w, o) : whole.next(c, p, w, o)) {
        const int u = o.hb * p.blocks + o.block;
        if (u < 0 || u >= units || (p.shared && o.unit != u)) { bad = "no such unit"; break; }
        if (o.part >= 0 && (o.part >= 2 * p.grid || o.part / 2 != w || slots[o.part]++)) bad = "a part's place";
        if (o.starts && w0[u] >= 0) bad = "two starts";
        if (o.ends && w1[u] >= 0) bad = "two ends";
        if (o.starts) w0[u] = w;
        if (o.ends) w1[u] = w;
        of[u].push_back(o);
        by[u].push_back(w);
        n += o.last > o.first ? o.last - o.first : 1;
      }
      most = n > most ? n : most;
      least = n < least ? n : least;
    }
    for (int u = 0; u < units && !bad; ++u) {
      int first, last, covered = 0;
      attn_tiles(c, u % p.blocks, &first, &last);
      if (of[u].empty() || w0[u] < 0 || w1[u] < w0[u]) { bad = "no start or end"; break; }
      if ((int)of[u].size() != w1[u] - w0[u] + 1) { bad = "number of parts"; break; }
      const bool parts = of[u].size() > 1;
      for (size_t i = 0; i < of[u].size(); ++i) {
        const AttnPiece& o = of[u][i];
        if ((o.part >= 0) != parts) bad = "a part or the whole";
        if (parts && (by[u][i] < w0[u] || by[u][i] > w1[u] || o.part != attn_part(w0[u], by[u][i]))) bad = "a part's owner";
        if (o.first < first || o.last > last) bad = "tiles outside";
        if (o.starts && o.first != first) bad = "the first part starts the unit";
        covered += o.last > o.first ? o.last - o.first : 0;
        for (size_t k = 0; k < i; ++k)
          if (o.first < of[u][k].last && of[u][k].first < o.last) bad = "tiles twice";
      }
      if (covered != (last > first ? last - first : 0)) bad = "tiles missing";
    }
    if (!bad && p.shared && most > least + 1) bad = "uneven shares";
    if (bad)
      printf("%s: held %lld passing %lld group %lld offset %lld causal %lld keys %lld heads %lld\n", bad, held, passing, group, offset,
             causal, by_keys, heads);
    else
      printf("ok %d %d\n", p.grid, p.shared);
  }
  return 0;
}
