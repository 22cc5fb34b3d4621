"""Calls of the experts' products, at least one for every shape of tiles."""

# (shape of matrices along k, of matrices across, experts, rows, k, n); sizes are whole
# units of 16 bytes in every type, but of the last two, whose rows are of any length
PRODUCTS = [
    ("Tiny", "FewAcross", 1, 5, 272, 208),
    ("Few", "FewAcross", 8, 9, 144, 2000),
    ("Few", "Low", 64, 100, 144, 1040),
    ("Low", "Low", 16, 256, 144, 1040),
    ("Some", "Some", 16, 480, 400, 1040),
    ("Middle", "Middle", 32, 1700, 144, 1040),
    ("Half", "Half", 32, 3000, 208, 2064),
    ("Large", "Large", 24, 5200, 144, 1040),
    ("AnyMiddle", "AnyMiddle", 16, 2000, 203, 1031),
    ("AnyFew", "AnyFew", 8, 100, 203, 331),
]
# (shape, experts, rows, n, k)
GRADIENTS = [
    ("Deep", 2, 2000, 136, 264),
    ("Middle", 12, 900, 776, 648),
    ("Large", 100, 4000, 392, 520),
    ("AnyMiddle", 12, 900, 391, 261),
]
