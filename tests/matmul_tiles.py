"""Sizes at which an NVFP4 product takes each tile width on 148 multiprocessors."""
# by words and one half, by words, by 16 bytes: how a row's K / 16 scales are read;
# all of them more than one turn of 4 steps
KS = (1184, 1344, 1280)
# (width, M, N)
DENSE = [(32, 33, 272), (32, 33, 1200), (64, 170, 3240), (64, 1590, 272), (128, 400, 3240),
         (192, 700, 4100), (192, 700, 4240), (224, 1590, 2192), (224, 2700, 4100)]
# (width, T, N, E)
GROUPED = [(32, 33, 1200, 3), (64, 170, 2100, 8), (128, 333, 2192, 8), (192, 700, 3104, 3),
           (192, 640, 3300, 3), (224, 900, 3240, 3), (224, 1590, 4100, 3)]
