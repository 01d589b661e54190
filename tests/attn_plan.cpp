// The attention kernels' deal of tiles to workgroups, on the host: for each
// line "held passing group offset causal by_keys heads block" of the input,
// every workgroup's part; prints "ok grid each" or what is wrong.
#include <stdio.h>

#include <vector>

#include "svdq_layout.h"

using namespace svdq;

int main() {
  long long held, passing, group, offset, causal, by_keys, heads, block;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &held, &passing, &group, &offset, &causal, &by_keys, &heads, &block) == 8) {
    const AttnCost c = {(int)held, (int)passing, (int)group, (int)offset, (int)causal, (int)by_keys, (int)block};
    const AttnPlan p = attn_plan(c, heads);
    const int units = p.blocks * (int)heads;
    const char* bad = nullptr;
    std::vector<int> seen(p.grid, 0), at(units, 0), count(units, 0);
    AttnParts deal;
    if (p.each) {
      if (p.grid > kAttnCus || units >= kAttnCus) bad = "more parts than run at once";
      else attn_parts(c, p, &deal);
    }
    int last_unit = -1;
    for (int id = 0; id < p.grid && !bad; ++id) {
      const int w = attn_place(p, id);
      if (w < 0 || w >= p.grid || seen[w]++) bad = "two workgroups at one place";
    }
    for (int w = 0; w < p.grid && !bad; ++w) {   // parts of a unit side by side, its tiles in order
      const AttnPiece o = p.each ? attn_piece(c, p, deal.at[w]) : attn_piece(c, p, w);
      const int u = o.hb * p.blocks + o.block;
      if (u < 0 || u >= units) { bad = "no such unit"; break; }
      int first, last;
      attn_tiles(c, o.block, &first, &last);
      if (p.each && (int)deal.at[w].part != count[u]) bad = "a part's number";
      if (p.each && count[u] == 0 && w > 0 && deal.at[w - 1].part != deal.at[w - 1].parts - 1) bad = "parts not side by side";
      if (o.starts != (count[u] == 0) || (count[u] == 0 && o.first != first)) bad = "the first part starts the unit";
      if (count[u] > 0 && (u != last_unit || o.first != at[u])) bad = "tiles not in order";
      if (o.last < o.first || o.last > last) bad = "tiles outside";
      if (p.each && o.last - o.first > p.each) bad = "a part too long";
      if (o.whole && (o.first != first || o.last != last)) bad = "not the whole";
      at[u] = o.last;
      ++count[u];
      last_unit = u;
    }
    for (int u = 0; u < units && !bad; ++u) {
      int first, last;
      attn_tiles(c, u % p.blocks, &first, &last);
      if (count[u] == 0 || at[u] != last) bad = "tiles missing";
    }
    if (p.each && !bad) {
      AttnJoins joins;
      int several = 0;
      const int n = attn_joins(p, deal, &joins);
      for (int u = 0; u < units; ++u) several += count[u] > 1;
      if (n != several || n == 0) bad = "units to join";
      for (int i = 0; i < n && !bad; ++i) {
        const AttnJoin j = joins.at[i];
        const AttnPiece o = attn_piece(c, p, deal.at[j.first]);
        if (o.hb * p.blocks + o.block != (int)j.unit || !o.starts || (int)j.parts != count[j.unit]) bad = "a unit to join";
      }
    }
    if (bad)
      printf("%s: held %lld passing %lld group %lld offset %lld causal %lld keys %lld heads %lld block %lld\n", bad, held, passing,
             group, offset, causal, by_keys, heads, block);
    else
      printf("ok %d %d\n", p.grid, p.each);
  }
  return 0;
}
