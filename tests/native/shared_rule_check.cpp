// Prints how w4a_attn_shared cuts the calls that it reads (compiled and run by
// tests/test_paged_paths.py; no GPU needed).  A line in: rows batch nq nkv hd
// page width P window max_new sms; a line out: few many with_prefix prefix_few
// ns_prefix ns_rest ns_own own_joins.
#include <cstdio>

#include "shared_rule.h"

int main() {
  int rows, batch, nq, nkv, hd, page, width, P, window, max_new, sms;
  while (scanf("%d %d %d %d %d %d %d %d %d %d %d", &rows, &batch, &nq, &nkv, &hd, &page, &width, &P, &window, &max_new,
               &sms) == 11) {
    const w4a::ShPlan p = w4a::shared_plan(rows, batch, nq, nkv, max_new, sms);
    const w4a::ShChoice c = w4a::shared_choice(p, batch, nkv, hd, page, width, P, window, max_new, sms);
    printf("%d %d %d %d %d %d %d %d\n", p.few, int(p.many), c.with_prefix, c.prefix_few, c.ns_prefix, c.ns_rest, c.ns_own,
           c.own_joins);
  }
  return 0;
}
