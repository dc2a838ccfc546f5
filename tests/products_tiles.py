"""Products by the kernel that they get: name -> (product, operands' type, rows of
each group, n, k, elements that the operands begin off a multiple of 16 bytes).
The name begins with the type, product, tile and whether the operands go straight
to LDS."""

CASES = {
    # up to one 128 x 128 tile per compute unit, at several counts
    "bf16 nt deep direct 144": ("nt", "bf16", [1100], 2040, 520, 0),
    "bf16 nt deep direct 224": ("nt", "bf16", [1700], 2040, 72, 0),
    "bf16 nt deep direct 256": ("nt", "bf16", [2048], 2048, 520, 0),
    "bf16 nt deep direct groups": ("nt", "bf16", [700, 0, 1, 900], 2056, 136, 0),
    "bf16 nt deep direct few rows": ("nt", "bf16", [37], 16520, 4104, 0),
    "bf16 nn deep direct 144": ("nn", "bf16", [1100], 2040, 520, 0),
    "bf16 nn deep direct 224": ("nn", "bf16", [1700], 2040, 72, 0),
    "bf16 nn deep direct 256": ("nn", "bf16", [2048], 2048, 520, 0),
    "bf16 nn deep direct groups": ("nn", "bf16", [700, 0, 1, 900], 2056, 136, 0),
    "bf16 tn deep direct 144": ("tn", "bf16", [520], 1096, 2040, 0),
    "bf16 tn deep direct 240": ("tn", "bf16", [333], 1800, 2040, 0),
    "bf16 tn deep direct 256": ("tn", "bf16", [520], 2048, 2048, 0),
    "bf16 tn deep direct groups": ("tn", "bf16", [200, 0, 131], 1032, 1032, 0),
}
