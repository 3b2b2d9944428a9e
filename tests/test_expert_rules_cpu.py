"""Which kernels the expert block's gate and up projection takes, at sizes where both forms were measured.  The measured times
(us of the whole call, streamed and tiled, one MI355X, two sets of weights in turn) stand with each case; the rule has to
take the faster form wherever they are 8% apart."""
import pytest

import ffn_rules as Rules

#  format, experts, hidden, intermediate, top-k, {rows per expert: (streamed, tiled)}
MEASURED = [
    ("bf16", 32, 7168, 256, 4, {4: (79, 139), 16: (97, 149), 32: (118, 164), 47: (139, 173)}),
    ("bf16", 32, 7168, 512, 4, {4: (134, 168), 16: (151, 182), 32: (172, 197), 47: (209, 206)}),
    ("bf16", 32, 7168, 768, 4, {4: (208, 196), 8: (222, 205), 16: (238, 217), 32: (237, 232), 47: (284, 245)}),
    ("bf16", 32, 7168, 1152, 4, {8: (297, 363), 16: (326, 372), 32: (350, 387), 47: (387, 400)}),
    ("bf16", 32, 7168, 1408, 4, {8: (352, 390), 16: (376, 400), 32: (421, 419), 47: (466, 435)}),
    ("bf16", 32, 7168, 1664, 4, {2: (350, 388), 16: (429, 436), 24: (458, 447), 32: (490, 459), 47: (539, 477)}),
    ("bf16", 32, 7168, 1792, 4, {8: (448, 436), 16: (463, 442), 32: (502, 469), 47: (564, 491)}),
    ("bf16", 64, 4096, 512, 4, {8: (176, 184), 16: (192, 193), 32: (217, 202), 47: (251, 216)}),
    ("bf16", 64, 4096, 1152, 4, {4: (331, 389), 16: (351, 412), 32: (389, 433), 47: (430, 453)}),
    ("bf16", 64, 4096, 1280, 4, {4: (384, 418), 16: (424, 440), 32: (484, 460), 47: (523, 482)}),
    ("bf16", 128, 2048, 640, 4, {4: (203, 229), 16: (222, 250), 32: (246, 265), 47: (278, 278)}),
    ("bf16", 128, 2048, 832, 4, {4: (252, 279), 16: (275, 304), 24: (289, 313), 47: (340, 340)}),
    ("fp8", 32, 8192, 384, 4, {4: (81, 97), 16: (91, 97), 32: (106, 105), 47: (119, 110)}),
    ("fp8", 32, 8192, 512, 4, {4: (102, 109), 16: (108, 113), 32: (121, 123), 47: (131, 131)}),
    ("fp8", 32, 8192, 640, 4, {4: (141, 123), 16: (151, 128), 32: (152, 137), 47: (168, 145)}),
    ("fp8", 32, 7168, 768, 4, {2: (117, 101), 8: (126, 107), 16: (147, 110), 32: (163, 120), 47: (165, 128)}),
    ("fp8", 32, 7168, 1152, 4, {2: (126, 114), 8: (177, 185), 16: (198, 198), 32: (216, 212), 47: (240, 218)}),
    ("fp8", 32, 7168, 1408, 4, {2: (171, 183), 8: (192, 206), 16: (221, 222), 24: (240, 227), 32: (256, 231), 47: (280, 238)}),
    ("fp8", 32, 7168, 1664, 4, {2: (188, 204), 8: (236, 226), 16: (261, 243), 24: (272, 248), 32: (294, 255), 47: (326, 263)}),
    ("fp8", 32, 7168, 1792, 4, {8: (244, 231), 16: (276, 250), 32: (309, 261), 47: (354, 272)}),
    ("fp8", 64, 4096, 640, 4, {4: (129, 140), 16: (139, 147), 32: (152, 156), 47: (162, 160)}),
    ("fp8", 64, 4096, 1152, 4, {4: (201, 211), 16: (211, 226), 32: (236, 237), 47: (255, 246)}),
    ("fp8", 64, 4096, 1280, 4, {4: (211, 221), 16: (232, 244), 32: (257, 256), 47: (286, 266)}),
    ("fp8", 64, 4096, 1408, 4, {4: (236, 235), 16: (249, 254), 32: (277, 266), 47: (305, 275)}),
    ("fp8", 128, 2048, 640, 4, {4: (116, 115), 16: (131, 122), 32: (147, 130), 47: (162, 136)}),
]
POINTS = [(f, E, H, I, K, rows, t) for f, E, H, I, K, times in MEASURED for rows, t in times.items()]


@pytest.mark.parametrize("fmt,E,H,I,K,rows,times", POINTS, ids=["%s-E%d-%dx%d-rows%d" % (p[0], p[1], p[2], p[3], p[5]) for p in POINTS])
def test_gate_and_up_takes_the_faster_form(fmt, E, H, I, K, rows, times):
    streamed, tiled = times
    took = streamed if Rules.path(rows * E // K, K, E, 1, H, I, fmt)[0] == "stream" else tiled
    assert took <= 1.08 * min(times), (took, times)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_more_rows_never_go_back_to_streaming(fmt):
    """From so many rows per expert on that weights are read once no longer by streaming, the tiles keep them (whole rounds of
    tiles: experts that get no row do not change the number)."""
    for I in (512, 1152, 1408, 1664, 2048):
        forms = [Rules.path(rows * 8, 4, 32, 1, 7168, I, fmt)[0] for rows in range(12, 64)]
        assert forms == sorted(forms), (I, forms)      # "stream" before "tile once"
