"""Sizes of the 4-bit LM head that reach each of its shapes: lone CTAs, pairs,
pairs that form two row tiles from one tile of W.  The library's own rule is
asked on the host (test_fp4_plan.py), so a retuned rule cannot leave one out."""

# (M, V, d): what is wanted of the rule
LONE = [(100, 3001, 2080), (64, 20000, 1568)]
PAIR = [(131, 40000, 1600), (200, 32003, 2080)]
# RT row tiles of 256: an even number, an odd one (whose last group has one tile), a vocabulary of no whole octets
TWO = [(257, 40000, 1600), (1280, 9000, 1824), (2304, 9728, 2048), (1030, 30001, 2080)]
ODD_LAST = [(1280, 9000, 1824), (2304, 9728, 2048), (1030, 30001, 2080)]
