/* Argument marshalling of the many-token and 8-bit calls, as a CPython module.
 *
 * Each function takes the C entry point's arguments (a tensor, an address or
 * None where it takes a pointer; a stream object, a handle or None, torch's
 * current stream, where it takes a stream) and returns its status.  A call
 * of a small batch is bound by the host: converting eight arguments here costs
 * about 0.3 us where the ctypes route costs 1.2.
 */
#include "binding.h"

ENTRY(smoe_topk_rows, 8, P(0); I(1); I(2); I(3); I(4); P(5); P(6); S(7), (p0, v1, v2, v3, v4, p5, p6, s))
ENTRY(smoe_topk_rows_backward, 8, P(0); P(1); P(2); I(3); I(4); I(5); P(6); S(7), (p0, p1, p2, v3, v4, v5, p6, s))
ENTRY(smoe_dispatch_tokens, 14, P(0); I(1); I(2); I(3); P(4); I(5); I(6); P(7); P(8); P(9); P(10); P(11); Z(12); S(13),
      (p0, v1, v2, v3, p4, v5, v6, p7, p8, p9, p10, p11, z12, s))
ENTRY(smoe_dispatch_tokens_backward, 8, P(0); I(1); P(2); I(3); I(4); I(5); P(6); S(7), (p0, v1, p2, v3, v4, v5, p6, s))
ENTRY(smoe_combine_tokens, 9, P(0); I(1); P(2); P(3); I(4); I(5); I(6); P(7); S(8), (p0, v1, p2, p3, v4, v5, v6, p7, s))
ENTRY(smoe_combine_tokens_backward, 11, P(0); P(1); I(2); P(3); P(4); I(5); I(6); I(7); P(8); P(9); S(10),
      (p0, p1, v2, p3, p4, v5, v6, v7, p8, p9, s))
ENTRY(smoe_quantize_rows_q8, 8, P(0); I(1); I(2); I(3); I(4); P(5); P(6); S(7), (p0, v1, v2, v3, v4, p5, p6, s))
ENTRY(smoe_matmul_q8, 12, P(0); P(1); I(2); P(3); P(4); I(5); I(6); P(7); I(8); P(9); Z(10); S(11),
      (p0, p1, v2, p3, p4, v5, v6, p7, v8, p9, z10, s))
ENTRY(smoe_experts_matmul_q8, 17,
      P(0); P(1); I(2); P(3); I(4); P(5); I(6); I(7); P(8); P(9); I(10); I(11); P(12); I(13); P(14); Z(15); S(16),
      (p0, p1, v2, p3, v4, p5, v6, v7, p8, p9, v10, v11, p12, v13, p14, z15, s))

static PyMethodDef methods[] = {
    FAST(smoe_topk_rows),
    FAST(smoe_topk_rows_backward),
    FAST(smoe_dispatch_tokens),
    FAST(smoe_dispatch_tokens_backward),
    FAST(smoe_combine_tokens),
    FAST(smoe_combine_tokens_backward),
    FAST(smoe_quantize_rows_q8),
    FAST(smoe_matmul_q8),
    FAST(smoe_experts_matmul_q8),
    BINDING_END,
};

BINDING_MODULE(_binding)
