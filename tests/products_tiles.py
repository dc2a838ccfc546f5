"""Products by the kernel that they get: name -> (product, operands' type, rows of
each group, n, k, elements that the operands begin off a multiple of 16 bytes).
The name begins with the type, product, tile and whether the operands go straight
to LDS."""

CASES = {
    # up to one 128 x 128 tile per compute unit, at several counts
    "bf16 nt deep direct 144": ("nt", "bf16", [1100], 2040, 520, 0),
    "bf16 nt deep direct 224": ("nt", "bf16", [1700], 2040, 72, 0),
    "bf16 nt deep direct 256": ("nt", "bf16", [2048], 2048, 520, 0),
    "bf16 nt deep direct groups": ("nt", "bf16", [700, 0, 1, 900], 2056, 392, 0),
    "bf16 nt deep direct few rows": ("nt", "bf16", [37], 16520, 4104, 0),
    "bf16 nn deep direct 144": ("nn", "bf16", [1100], 2040, 520, 0),
    "bf16 nn deep direct 224": ("nn", "bf16", [1700], 2040, 72, 0),
    "bf16 nn deep direct 256": ("nn", "bf16", [2048], 2048, 520, 0),
    "bf16 nn deep direct groups": ("nn", "bf16", [700, 0, 1, 900], 2056, 392, 0),
    "bf16 tn deep direct 144": ("tn", "bf16", [520], 1096, 2040, 0),
    "bf16 tn deep direct 240": ("tn", "bf16", [333], 1800, 2040, 0),
    "bf16 tn deep direct 256": ("tn", "bf16", [520], 2048, 2048, 0),
    "bf16 tn deep direct groups": ("tn", "bf16", [1600, 0, 131], 1032, 1032, 0),
}

for _op in ("nt", "nn"):
    CASES.update({
        f"bf16 {_op} thin direct": (_op, "bf16", [7, 0, 30, 1, 2], 200, 1096, 0),
        f"bf16 {_op} apart direct": (_op, "bf16", [70, 0, 200, 1, 300], 328, 4104, 0),
        # 64 x 64 tiles: few rows over experts, and groups that end inside a tile
        f"bf16 {_op} small direct experts": (_op, "bf16", [2] * 8, 2048, 512, 0),
        f"bf16 {_op} small direct groups": (_op, "bf16", [200, 1, 0, 70, 500], 1032, 264, 0),
        f"bf16 {_op} small direct one round": (_op, "bf16", [777], 1352, 8, 0),
        f"bf16 {_op} small direct five": (_op, "bf16", [777], 1352, 296, 0),
        f"bf16 {_op} mid direct": (_op, "bf16", [700, 0, 1, 1400], 2056, 72, 0),
        f"bf16 {_op} big direct": (_op, "bf16", [2600, 3, 0, 1900], 4104, 200, 0),
        f"bf16 {_op} small registers": (_op, "bf16", [200, 1, 0, 70], 137, 265, 0),
        f"bf16 {_op} mid registers": (_op, "bf16", [700, 0, 1, 1400], 2051, 70, 1),
        f"i8 {_op} thin direct": (_op, "i8", [7, 0, 30, 1, 2], 200, 1096, 0),
        f"i8 {_op} apart direct": (_op, "i8", [70, 0, 200, 1, 300], 329, 5001, 0),
        f"i8 {_op} small direct experts": (_op, "i8", [2] * 8, 2048, 512, 0),
        f"i8 {_op} small direct groups": (_op, "i8", [300, 77, 400], 1025, 2049, 0),
        f"i8 {_op} small direct one round": (_op, "i8", [777], 1350, 100, 0),
        f"i8 {_op} mid direct": (_op, "i8", [700, 0, 1, 1400], 2051, 70, 0),
        f"i8 {_op} big direct": (_op, "i8", [2600, 3, 0, 1900], 4104, 200, 0),
        f"f32 {_op} tiny registers": (_op, "f32", [200, 1, 0, 70], 137, 265, 0),
        f"f32 {_op} small registers": (_op, "f32", [700, 0, 1, 800], 1480, 70, 0),
        f"f32 {_op} small registers 1": (_op, "f32", [1500], 1401, 133, 1),
        f"f32 {_op} mid registers": (_op, "f32", [700, 0, 1, 1400], 2051, 70, 1),
    })
CASES.update({
    "bf16 tn small direct": ("tn", "bf16", [200, 1, 0, 70], 136, 264, 0),
    "bf16 tn mid direct": ("tn", "bf16", [70, 61], 2056, 2120, 0),
    "bf16 tn big direct one": ("tn", "bf16", [300], 4096, 4096, 0),
    "bf16 tn big direct groups": ("tn", "bf16", [137, 9], 4104, 4104, 0),
    "bf16 tn small registers": ("tn", "bf16", [200, 1, 0, 70], 137, 265, 0),
    "bf16 tn mid registers": ("tn", "bf16", [70, 61], 2051, 2118, 1),
    "f32 tn tiny registers": ("tn", "f32", [200, 1, 0, 70], 137, 265, 0),
    "f32 tn small registers": ("tn", "f32", [333], 1500, 1401, 1),
    "f32 tn small registers groups": ("tn", "f32", [200, 0, 70], 840, 840, 0),
    "f32 tn mid registers": ("tn", "f32", [70, 61], 2051, 2050, 1),
})
