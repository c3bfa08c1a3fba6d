"""Bounds of the relative 2-norm tests of linear attention, and that norm."""
# Bounds on the relative 2-norm of a whole output, where the errors of its entries average instead of adding up as in
# linear_testlib's ``check``.  They are near the stated accuracy, so that a part that a product leaves out shows (test_linear_accuracy.py
# plants that in the oracle):
# FP32_NORM  states and their gradients, everything of an fp32 call.  Three bf16 parts leave 2^-24 of a term, three tf32
#            products 2^-22; the sums of the rows that matter take up to 24 matrix steps, each of which truncates up to
#            2^-23 of the sum so far, in the mean half of it from a sum half as large: 24 2^-25 < 2^-20.
# TWO_PART_NORM  gradients of the decays in a bf16 call: the state, its gradient and their product with two parts each,
#            three independent errors of at most 2^-17: sqrt(3) 2^-17 < 2^-16.
# BF16_NORM  bf16 outputs: the output's rounding and one operand's, each at most 2^-8 and evenly spread (1 / sqrt(3) of it
#            in the mean of the squares): sqrt(2 / 3) 2^-8.
FP32_NORM = 2.0 ** -20
TWO_PART_NORM = 2.0 ** -16
BF16_NORM = (2.0 / 3.0) ** 0.5 * 2.0 ** -8


def relative(got, ref):
    got, ref = got.detach().cpu().double(), ref.double()
    return ((got - ref).norm() / ref.norm()).item()
