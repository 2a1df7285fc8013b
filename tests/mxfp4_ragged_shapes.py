"""SwiGLU calls of the microscaled 4-bit path whose outputs end inside a block of columns: a CPU test
holds them to the host's choice of kernel, the GPU tests run them."""

# (answer of the host's choice): n, d, lengths of the segments
RAGGED = [("rows 1 4", (2, 96, [1, 2, 0, 1])), ("rows 1 4", (2 * 49, 1056, [1, 4, 0, 2, 1, 1])),
          ("rows 1 2", (2 * 2035, 1056, [3, 1, 1, 0, 2, 2, 1, 1, 1])), ("rows 2 2", (2 * 77, 544, [4, 3, 17])),
          ("rows 2 2", (2 * 31, 32, [7, 1, 3])), ("tile 64", (2 * 301, 1056, [70, 0, 130, 257, 3])),
          ("tile 64", (2 * 65, 288, [64, 1, 33, 0, 16])), ("tile 64", (2, 160, [70, 1])),
          ("tile 256", (2 * 4101, 544, [300, 0, 100, 260, 40])), ("tile 256", (2 * 10241, 96, [129, 65]))]
