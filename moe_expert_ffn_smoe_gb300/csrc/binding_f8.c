/* Argument marshalling of the calls for routing by scores, 8-bit floating point and
 * the weights' gradient, as binding.c does it for the calls that were there before. */
#include "binding.h"

ENTRY(smoe_route_rows, 15,
      P(0); I(1); I(2); I(3); P(4); I(5); I(6); I(7); I(8); I(9); I(10); F(11); P(12); P(13); S(14),
      (p0, v1, v2, v3, p4, v5, v6, v7, v8, v9, v10, f11, p12, p13, s))
ENTRY(smoe_route_rows_backward, 13, P(0); I(1); I(2); I(3); I(4); I(5); I(6); F(7); P(8); P(9); P(10); P(11); S(12),
      (p0, v1, v2, v3, v4, v5, v6, f7, p8, p9, p10, p11, s))
ENTRY(smoe_quantize_rows_f8, 8, P(0); I(1); I(2); I(3); I(4); P(5); P(6); S(7), (p0, v1, v2, v3, v4, p5, p6, s))
ENTRY(smoe_quantize_blocks_f8, 10, P(0); I(1); I(2); I(3); I(4); P(5); P(6); P(7); P(8); S(9),
      (p0, v1, v2, v3, v4, p5, p6, p7, p8, s))
ENTRY(smoe_matmul_f8, 12, P(0); P(1); I(2); P(3); P(4); I(5); I(6); P(7); I(8); P(9); Z(10); S(11),
      (p0, p1, v2, p3, p4, v5, v6, p7, v8, p9, z10, s))
ENTRY(smoe_experts_matmul_f8, 17,
      P(0); P(1); I(2); P(3); I(4); P(5); I(6); I(7); P(8); P(9); I(10); I(11); P(12); I(13); P(14); Z(15); S(16),
      (p0, p1, v2, p3, v4, p5, v6, v7, p8, p9, v10, v11, p12, v13, p14, z15, s))
ENTRY(smoe_experts_weight_grad, 11, P(0); P(1); P(2); I(3); I(4); I(5); I(6); I(7); P(8); I(9); S(10),
      (p0, p1, p2, v3, v4, v5, v6, v7, p8, v9, s))

static PyMethodDef methods[] = {
    FAST(smoe_route_rows),
    FAST(smoe_route_rows_backward),
    FAST(smoe_quantize_rows_f8),
    FAST(smoe_quantize_blocks_f8),
    FAST(smoe_matmul_f8),
    FAST(smoe_experts_matmul_f8),
    FAST(smoe_experts_weight_grad),
    BINDING_END,
};

BINDING_MODULE(_binding_f8)
