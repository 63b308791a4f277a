"""Sizes (tokens, in, out) of the layer above 16 tokens for each form of its
kernel: one tile per cluster whose pairs split the channels ("split"), and
clusters that walk many tiles ("whole")."""

SPLIT = [(17, 512, 272), (50, 512, 272), (64, 2560, 1040), (128, 512, 272), (100, 1536, 528), (300, 768, 400),
         (700, 512, 656), (40, 384, 18928), (100, 384, 18928)]
WHOLE = [(513, 384, 272), (2000, 384, 8192), (4000, 512, 4112), (1500, 768, 9728), (333, 256, 17424), (129, 128, 37888)]
