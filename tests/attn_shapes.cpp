// What the attention kernels' launches take for granted of their plans: for
// each line "samples queries keys heads kv_heads head_dim causal scaled" of the
// input both passes; prints "ok" and the launch of each or what is wrong.
#include <stdio.h>

#include "svdq_layout.h"

using namespace svdq;

static const char* check(const AttnCost& c, const AttnPlan& p, int64_t D, bool keys) {
  if (c.block != 4 * kAttnWave && c.block != 8 * kAttnWave) return "neither four nor eight waves";
  if (c.ways != 1 && c.ways != 2) return "neither one nor two ways";
  if (c.ways == 2 && c.block != 4 * kAttnWave) return "two ways of eight waves";
  if (c.fine != (D <= 32 || c.held <= kAttnTile || c.passing <= kAttnTile)) return "operands a probability";
  if (c.fine && D > 32 && (c.block != 8 * kAttnWave || c.ways != 1)) return "two operands without eight waves";
  if (keys && D > 96 && c.block != 8 * kAttnWave) return "keys of large heads without eight waves";
  if (p.each && c.block == 4 * kAttnWave && c.ways == 1) return "parts of workgroups that take none";
  if (p.each && p.grid > kAttnCus) return "more parts than run at once";
  if (!p.each && p.grid != p.blocks * p.heads) return "not a workgroup a unit";
  return nullptr;
}

int main() {
  long long B, Lq, Lk, H, Hk, D, causal, scaled;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &B, &Lq, &Lk, &H, &Hk, &D, &causal, &scaled) == 8) {
    const AttnSizes s = {B, Lq, Lk, H, Hk, D, causal != 0, scaled != 0};
    const AttnWs f = attn_ws(s);
    const AttnGradWs g = attn_grad_ws(s);
    const char* bad = check(f.cost, f.plan, D, false);
    if (!bad) bad = check(g.rows, g.dq, D, false);
    if (!bad) bad = check(g.keys, g.dkv, D, true);
    if (!bad && (int64_t)g.dq.blocks * g.rows.block % kAttnTile) bad = "rows up to a part of a tile";
    const int G = (int)(H / Hk), rows = (int)(Lq * G);
    const AttnGroup group = attn_group(G);
    for (int r : {0, 1, G - 1, G, rows - 1, rows, (1 << 30) - 1, (1 << 30) / G * G - 1 + (G == 1), 0x2aaaaaaa, 0x3fedcba9})
      if (!bad && r >= 0 && r < 1 << 30 && attn_query(group, r) != r / G) bad = "the query of a row";
    if (bad)
      printf("%s: %lld %lld %lld %lld %lld %lld %lld %lld\n", bad, B, Lq, Lk, H, Hk, D, causal, scaled);
    else
      printf("ok %d/%d/%d %d/%d/%d\n", f.cost.block / kAttnWave, f.cost.ways, f.plan.each > 0, g.keys.block / kAttnWave, g.keys.ways,
             g.dkv.each > 0);
  }
  return 0;
}
