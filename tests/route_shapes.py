"""Shapes that between them send the 4-bit product and the gated projection
through every kernel, tile and way of cutting that their host routes choose
among (on 256 compute units).  test_route_shapes_cpu.py asks the routes
themselves; the GPU tests run the shapes."""

# (matrices, weight panels, token panels, tiles over all of k, k in parts) of
# q4_route -> n, k, m.  Weight panels 8 is the kernel that shares activations, 16
# the LDS-fed tiles.
Q4 = {
    (1, 8, 1, False, False): (129, 300, 21),
    (1, 8, 1, False, True): (37, 1030, 9),
    (1, 8, 2, False, False): (4097, 515, 203),
    (1, 8, 2, False, True): (5, 3100, 701),
    (1, 8, 4, False, False): (1100, 33, 901),
    (1, 8, 4, False, True): (1100, 2100, 301),
    (1, 16, 8, True, False): (4097, 515, 1003),
    (1, 16, 8, False, True): (6000, 4100, 101),
    (1, 16, 8, True, True): (8200, 515, 901),
    (1, 16, 16, True, False): (8201, 5, 901),
    (1, 16, 16, False, True): (8200, 3100, 401),
    (1, 16, 16, True, True): (4100, 12000, 4096),
    (2, 8, 1, False, False): (300, 257, 21),
    (2, 8, 1, False, True): (37, 1030, 9),
    (2, 8, 2, False, False): (4097, 515, 203),
    (2, 8, 2, False, True): (5, 1030, 1601),
    (2, 8, 4, False, False): (1100, 33, 901),
    (2, 8, 4, False, True): (1100, 2100, 301),
    (2, 16, 8, True, False): (5003, 260, 2101),
    (2, 16, 8, False, True): (6000, 2600, 101),
    (2, 16, 8, True, True): (12003, 515, 333),
    (2, 16, 16, True, False): (5000, 260, 1003),
    (2, 16, 16, False, True): (2300, 3100, 901),
    (2, 16, 16, True, True): (20550, 4100, 400),
}
# Rows of fewer than eight columns go to the tiles whatever the tokens.
Q4_NARROW = [(48, 5, 9), (129, 7, 300), (300, 1, 33)]

# (token panels, tiles over all of k, k in parts) of the forward plan -> n, k, m
GATED_FORWARD = {
    (4, True, False): (320, 192, 133),
    (4, False, True): (64, 768, 129),
    (4, True, True): (1024, 1536, 2050),
    (8, True, False): (12800, 64, 131),
    (8, False, True): (2816, 4096, 201),
    (8, True, True): (6400, 768, 1301),
    (16, True, False): (10240, 64, 401),
    (16, False, True): (10240, 4096, 201),
    (16, True, True): (12800, 1024, 701),
}
# (token panels of dX, dX and dW in one launch, small dW tiles, dX in parts) of
# the plan of all gradients -> n, k, m
GATED_BACKWARD = {
    (4, True, True, False): (64, 64, 129),
    (4, True, True, True): (320, 64, 131),
    (4, False, True, False): (64, 4096, 901),
    (4, False, True, True): (5120, 64, 520),
    (4, False, False, True): (2816, 4096, 261),
    (8, True, True, False): (64, 2048, 2050),
    (8, True, True, True): (2816, 1024, 333),
    (8, False, True, False): (192, 4096, 1030),
    (8, False, True, True): (8192, 64, 521),
    (8, False, False, True): (3200, 2560, 261),
    (8, False, False, False): (1024, 10240, 520),
    (16, True, True, False): (64, 4096, 2050),
    (16, True, True, True): (6400, 64, 1301),
    (16, False, True, False): (192, 4096, 2050),
    (16, False, True, True): (8192, 64, 1030),
    (16, False, False, True): (3200, 2560, 401),
    (16, False, False, False): (2816, 4096, 2051),
}
