"""Sizes for each form of the 8-bit product's kernel, on a GPU of 152 SMs that runs 76 pairs of CTAs at once: (form, rows of
every expert, columns of the result, columns of the rows, padding behind each row, transposed)."""
FEW_ROWS, COLUMNS_128, COLUMNS_256, PAIRS = range(4)

FORM_CASES = [(FEW_ROWS, [0, 1, 5], 528, 1040, 0, False), (FEW_ROWS, [3, 0, 2], 512, 1024, 0, False), (FEW_ROWS, [8], 1008, 256, 16, False)]
for _t in (False, True):
    FORM_CASES += [
        (COLUMNS_128, [5, 130, 0, 7], 528, 400, 0, _t), (COLUMNS_128, [40, 200, 0, 129], 512, 384, 0, _t),
        (COLUMNS_256, [130] * 30 + [0, 1, 128, 127, 300] * 2, 1040, 144, 0, _t), (COLUMNS_256, [130] * 30 + [0, 1, 128, 127, 300] * 2, 1792, 256, 0, _t),
        (PAIRS, [2299], 2048, 256, 0, _t), (PAIRS, [2299], 2048, 400, 0, _t), (PAIRS, [1100, 0, 1190], 1536, 256, 16, _t),
        (PAIRS, [129, 1, 256, 4700, 40], 4112, 80, 0, _t)]
