"""Matrices whose products take tiles of 64, 128 and 256, with sides that none
of them divides: ((rows, cols) of equal matrices, how many, the side of the
symmetric products' tiles, that of the products with X)."""
TILES = [((300, 500), 2, 64, 64), ((1300, 2100), 1, 64, 128), ((700, 900), 12, 128, 128), ((131, 2083), 23, 64, 256),
         ((1025, 1030), 30, 128, 256), ((901, 903), 25, 256, 256)]
