"""Sizes of the gated feed-forward block whose products take tiles of 256 x 256
everywhere (tokens, features, columns of x): ends inside a tile and a step in all
three, fewer features than columns, and whole ones."""
LARGE = [(4090, 2044, 4072), (3000, 1500, 2504), (4096, 2048, 4096)]
